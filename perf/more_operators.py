"""Cases, inputs and plain forms of the gated block's training and of 4-bit weights.

The block in question is the first half of a gated FFN, h = A(x W1^T) * (x W3^T):

* ``gated_up`` -- h from bf16 weights, for one token up to a prompt, and differentiable:
  a training step returns h and the gradients of x, W1 and W3;
* ``quantize_int4`` / ``dequantize_int4`` -- 4-bit codes of a weight matrix, two a byte,
  with a scale per group of columns (or per row), and the values they stand for;
* ``matmul_int4`` -- bf16 tokens by 4-bit weights;
* ``gated_up_int4`` -- h from 4-bit weights.

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
        # an up projection of the D = 2560 layer into 4 bits, a scale per 64 columns, and back
        {"name": "codes_up", "op": "codes", "N": 7168, "K": 2560, "group": 64, "out": "bf16"},
        # a down projection of the D = 4096 layer, one scale per output channel (group 0), its values kept in fp32
        {"name": "codes_down", "op": "codes", "N": 4096, "K": 14336, "group": 0, "out": "f32"},
        # one decoded token through a 4-bit up projection
        {"name": "int4_token", "op": "int4", "T": 1, "N": 7168, "K": 2560, "group": 64, "out": "bf16"},
        # an odd decode batch through its 4-bit down projection (few output rows, a long sum), fp32 out
        {"name": "int4_batch", "op": "int4", "T": 13, "N": 2560, "K": 7168, "group": 0, "out": "f32"},
        # a prompt batch through a 4-bit up projection of the D = 4096 layer
        {"name": "int4_prompt", "op": "int4", "T": 2048, "N": 14336, "K": 4096, "group": 64, "out": "bf16"},
        # one decoded token through the 4-bit gated block of a cast layer (90 % of the gate dead)
        {"name": "gated4_token", "op": "gated4", "T": 1, "D": 2560, "H": 7168, "group": 64, "act": "relu"},
        # a decode batch through the wide layer's, with the smooth gate
        {"name": "gated4_batch", "op": "gated4", "T": 24, "D": 4096, "H": 14336, "group": 128, "act": "silu"},
        # one decoded token through the bf16 gated block of a cast layer
        {"name": "gated_token", "op": "gated", "T": 1, "D": 2560, "H": 7168, "act": "relu"},
        # a prompt batch through it
        {"name": "gated_prompt", "op": "gated", "T": 4096, "D": 2560, "H": 7168, "act": "rsp"},
        # a training step of a small layer on an odd batch (rows and hidden units that fill no tile)
        {"name": "train_small", "op": "train", "T": 77, "D": 384, "H": 1000, "act": "silu"},
        # a training step of one fine-grained expert's share of a batch
        {"name": "train_expert", "op": "train", "T": 1000, "D": 2560, "H": 1024, "act": "rsp"},
        # a training step of the D = 2560 layer being cast, a full batch of tokens
        {"name": "train_cast", "op": "train", "T": 8192, "D": 2560, "H": 7168, "act": "relu"},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number spread over the logarithm of [lo, hi], a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + step)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    most = work({"op": "train", "T": 8192, "D": 2560, "H": 7168, "act": "relu"})["flops"]
    while True:
        op = rng.choice(("codes", "int4", "gated4", "gated", "train"))
        group = rng.choice((0, 64, 64, 128, 256))
        act = rng.choice(("relu", "rsp", "silu"))
        if op == "codes":
            c = {"op": op, "N": _log(rng, 1, 14336), "K": _log(rng, 64, 14336, 16), "group": group,
                 "out": rng.choice(("bf16", "f32"))}
        elif op == "int4":
            c = {"op": op, "T": _log(rng, 1, 2048), "N": _log(rng, 16, 14336), "K": _log(rng, 64, 14336, 16),
                 "group": group, "out": rng.choice(("bf16", "f32"))}
        elif op == "gated4":
            c = {"op": op, "T": _log(rng, 1, 1024), "D": _log(rng, 64, 4096, 16), "H": _log(rng, 16, 14336),
                 "group": group, "act": act}
        elif op == "gated":
            c = {"op": op, "T": _log(rng, 1, 4096), "D": _log(rng, 64, 4096, 8), "H": _log(rng, 16, 14336), "act": act}
        else:
            c = {"op": op, "T": _log(rng, 1, 8192), "D": _log(rng, 64, 4096, 8), "H": _log(rng, 16, 14336), "act": act}
        if work(c)["flops"] <= most:
            return c


def _groups(K, group):
    """Columns a scale covers, and scales a row."""
    size = group or K
    return size, -(-K // size)


def work(case):
    op = case["op"]
    if op == "codes":
        N, K = case["N"], case["K"]
        # the weights in, their values and scales out; a maximum, a quotient and a product for each
        return {"bytes": N * K * (2 + (2 if case["out"] == "bf16" else 4)) + N * _groups(K, case["group"])[1] * 4,
                "flops": 3 * N * K}
    if op == "int4":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": T * K * 2 + N * K // 2 + N * _groups(K, case["group"])[1] * 4
                + T * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * T * N * K}
    T, D, H = case["T"], case["D"], case["H"]
    # of W3 the rows of units that are live for some token (10 % of a token's units with the shifted ReLU and R-S+ gates,
    # all with SiLU); a tile of many tokens has no dead unit, so the operations are the dense formula's
    live = 1.0 if case["act"] == "silu" else 1 - 0.9 ** T
    flops = 4 * T * D * H * (1.0 if T > 8 else (1 + live) / 2)
    if op == "gated4":
        row = D / 2 + _groups(D, case["group"])[1] * 4
        return {"bytes": T * D * 2 + H * row * (1 + live) + T * H * 2, "flops": flops}
    if op == "gated":
        return {"bytes": T * D * 2 + H * D * 2 * (1 + live) + T * H * 2, "flops": flops}
    # x, the weights and dh in, h and the three gradients out; two products forward and four backward
    return {"bytes": T * D * 4 + H * D * 8 + T * H * 4, "flops": 12 * T * D * H}


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 2654435761 % (1 << 62) + 29)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _padded(w, group):
    """w [N, K] in fp32 as [N, groups, columns of a group], the last group filled up with zeros."""
    size, n = _groups(w.shape[1], group)
    p = torch.zeros(w.shape[0], n * size, device=w.device)
    p[:, :w.shape[1]] = w.float()
    return p.view(w.shape[0], n, size)


def _int4(w, group):
    """Codes [N, K] in -7 .. 7 and scales [N, groups] fp32: s = max|w| / 7 of a group, code = w / s to even."""
    p = _padded(w, group)
    amax = p.abs().amax(2)
    scale = amax / torch.full_like(amax, 7)  # a tensor on both sides: the correctly rounded quotient
    q = p / torch.where(scale > 0, scale, torch.ones_like(scale))[:, :, None]
    return q.round_().clamp_(-7, 7).view(w.shape[0], -1)[:, :w.shape[1]], scale


def _packed(q):
    """Two codes a byte, two's complement, the even column in the low nibble."""
    n = q.to(torch.int32) & 15
    return (n[:, 0::2] | n[:, 1::2] << 4).to(torch.uint8)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case, "group": case.get("group") or None}
    if op == "codes":
        w = _randn(g, case["N"], case["K"], dtype=BF)
        w *= case["K"] ** -0.5
        if case["N"] > 2:
            w[case["N"] // 2] = 0  # a pruned channel
        s["w"] = w
    elif op == "int4":
        s["x"] = _randn(g, case["T"], case["K"], dtype=BF)
        q, s["sw"] = _int4(_randn(g, case["N"], case["K"], dtype=BF) * case["K"] ** -0.5, case["group"])
        s["wq"] = _packed(q)
    else:
        T, D, H = case["T"], case["D"], case["H"]
        x = _randn(g, T, D, dtype=BF)
        x[:, -1] = 1
        W1, W3 = _randn(g, H, D, dtype=BF), _randn(g, H, D, dtype=BF)
        W1 *= D ** -0.5
        W3 *= D ** -0.5
        if case["act"] != "silu":
            W1[:, -1] = SHIFT  # the gate's bias, carried by the channel that is 1
        if op == "gated4":
            s["x"] = x
            for name, w in (("1", W1), ("3", W3)):
                q, s["s" + name] = _int4(w, case["group"])
                s["w" + name] = _packed(q)
        else:
            s.update(x=x, W1=W1, W3=W3)
            if op == "train":
                for name in ("x", "W1", "W3"):
                    s[name].requires_grad_()
                s["dh"] = _randn(g, T, H, dtype=BF)
    return s


# ---------------------------------------------------------------- the plain forms


def _values(codes, scales, K, group):
    """The matrix [N, K] in fp32 that packed codes and their scales stand for."""
    size, n = _groups(K, group)
    low, high = (codes & 15).to(torch.int8), (codes >> 4).to(torch.int8)
    q = torch.stack((low, high), 2).view(codes.shape[0], K)
    q = torch.where(q > 7, q - 16, q).float()
    return q * scales.repeat_interleave(size, 1)[:, :K]


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    v = z / (1 + torch.exp(-z))
    return v if act == "silu" else torch.where(z > 0, v, torch.zeros_like(v))


def _slope(z, act):
    if act == "relu":
        return (z > 0).float()
    p = 1 / (1 + torch.exp(-z))
    v = p * (1 + z * (1 - p))
    return v if act == "silu" else torch.where(z > 0, v, torch.zeros_like(v))


def _plain(s):
    c = s["case"]
    op = c["op"]
    out = torch.float32 if c.get("out") == "f32" else BF
    if op == "codes":
        q, scale = _int4(s["w"], c["group"])
        return (q * scale.repeat_interleave(_groups(c["K"], c["group"])[0], 1)[:, :c["K"]]).to(out), scale
    x = s["x"].detach().float()
    if op == "int4":
        return (x @ _values(s["wq"], s["sw"], c["K"], c["group"]).T).to(out)
    if op == "gated4":
        z = x @ _values(s["w1"], s["s1"], c["D"], c["group"]).T
        return (_act(z, c["act"]) * (x @ _values(s["w3"], s["s3"], c["D"], c["group"]).T)).to(BF)
    W1, W3 = s["W1"].detach().float(), s["W3"].detach().float()
    z, u = x @ W1.T, x @ W3.T
    a = _act(z, c["act"])
    h = (a * u).to(BF)
    if op == "gated":
        return h
    dh = s["dh"].float()
    dz, du = dh * u * _slope(z, c["act"]), dh * a
    return h, (dz @ W1 + du @ W3).to(BF), (dz.T @ x).to(BF), (du.T @ x).to(BF)


def run(state):
    if not own:
        return _plain(state)
    import activation_sparse_gated_gb300 as sffn
    c = state["case"]
    op = c["op"]
    if op == "codes":
        codes, scales = sffn.quantize_int4(state["w"], group=state["group"])
        return sffn.dequantize_int4(codes, scales, group=state["group"], dtype=c["out"]), scales
    if op == "int4":
        return sffn.matmul_int4(state["x"], state["wq"], state["sw"], group=state["group"], dtype=c["out"])
    if op == "gated4":
        return sffn.gated_up_int4(state["x"], state["w1"], state["s1"], state["w3"], state["s3"], group=state["group"],
                                  act=c["act"])
    h = sffn.gated_up(state["x"], state["W1"], state["W3"], act=c["act"])
    if op == "gated":
        return h
    return (h.detach(), *torch.autograd.grad(h, (state["x"], state["W1"], state["W3"]), state["dh"]))


# ---------------------------------------------------------------- the definitions in 64 bits


def _meant(codes, scales, K, group):
    """What packed codes and scales stand for, in 64 bits: a byte's two codes by a table, then each group's columns."""
    pair = torch.tensor([[(b & 15) - 16 * ((b & 15) > 7), (b >> 4) - 16 * ((b >> 4) > 7)] for b in range(256)],
                        dtype=torch.float64, device=codes.device)
    w = pair[codes.long()].reshape(codes.shape[0], K)
    size = group if group else K
    for j in range(scales.shape[1]):
        w[:, j * size:(j + 1) * size] *= scales[:, j:j + 1].double()
    return w


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "codes":
        # scales are held in binary32 and the codes are decided in it, by definition; the value is their product
        w = s["w"].float().cpu().numpy()
        f32, size = w.dtype.type, case["group"] or case["K"]
        values, scales = [], []
        for k in range(0, case["K"], size):
            part = w[:, k:k + size]
            scale = (abs(part).max(1) / f32(7))[:, None]
            q = (part / (scale + (scale == 0))).round().clip(-7, 7)
            values.append(torch.from_numpy(q).double() * torch.from_numpy(scale).double())
            scales.append(torch.from_numpy(scale))
        return torch.cat(values, 1), torch.cat(scales, 1)
    x = s["x"].detach().double()
    if op == "int4":
        return x @ _meant(s["wq"], s["sw"], case["K"], case["group"]).T
    if op == "gated4":
        W1, W3 = (_meant(s["w" + i], s["s" + i], case["D"], case["group"]) for i in "13")
    else:
        W1, W3 = s["W1"].detach().double(), s["W3"].detach().double()
    z, u = x @ W1.T, x @ W3.T
    p = torch.sigmoid(z)
    on = z > 0
    if case["act"] == "relu":
        gate, slope = z * on, on.double()
    else:
        gate, slope = z * p, p + z * p * torch.sigmoid(-z)
        if case["act"] == "rsp":
            gate, slope = gate * on, slope * on
    if op != "train":
        return gate * u
    dh = s["dh"].double()
    du = dh * gate
    dz = dh * slope * u
    return gate * u, torch.cat((dz, du), 1) @ torch.cat((W1, W3), 0), dz.T @ x, du.T @ x
