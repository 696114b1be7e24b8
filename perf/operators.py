"""Measured cases of the routing operators (moe_topk_route and its backward
pass), the 8-bit integer expert product (moe_int8_product) and the combine of
any k (moe_combine_topk), each with its plain form in torch operations.

With ``own`` false ``run`` computes the plain form; with ``own`` true it calls
the library. ``exact`` computes the same outputs in 64 bits from the formulas.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "i8": torch.int8}
FLT_MAX = 3.4028234663852886e38
BYTES = {"f32": 4, "bf16": 2, "i8": 1}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # One token of the 8-expert, top-2 layer: the latency of routing a single decode step.
        {"name": "route one token", "kind": "route", "T": 1, "E": 8, "k": 2, "type": "f32", "score": "softmax",
         "groups": 1, "keep": 1, "rule": "max", "bias": False, "renorm": False, "scale": 1.0, "valid": 1, "mask": 0.0},
        # A decode batch padded to a captured graph's 64 rows, many small experts in groups, balance bias.
        {"name": "route decode padded", "kind": "route", "T": 64, "E": 256, "k": 8, "type": "bf16", "score": "sigmoid",
         "groups": 8, "keep": 4, "rule": "top2", "bias": True, "renorm": True, "scale": 2.5, "valid": 57, "mask": 0.0},
        # A long prefill of the same router.
        {"name": "route prefill", "kind": "route", "T": 16384, "E": 256, "k": 8, "type": "f32", "score": "sigmoid",
         "groups": 8, "keep": 4, "rule": "top2", "bias": True, "renorm": True, "scale": 2.5, "valid": 16384, "mask": 0.0},
        # Router training at the 8-expert shape: one micro-batch of the sublayer.
        {"name": "route grad 8 experts", "kind": "route_grad", "T": 4096, "E": 8, "k": 2, "type": "f32",
         "score": "softmax", "renorm": True, "scale": 1.0, "valid": 4096, "mask": 0.0, "scores": False},
        # Router training with many experts and a balance loss on the scores.
        {"name": "route grad 256 experts", "kind": "route_grad", "T": 16384, "E": 256, "k": 8, "type": "bf16",
         "score": "sigmoid", "renorm": True, "scale": 2.5, "valid": 16384, "mask": 0.0, "scores": True},
        # Decode at the Grok-1 shape, T = 64: gate and up projections of 128 rows gathered from 64 tokens.
        {"name": "int8 gate/up decode", "kind": "product", "R": 128, "K": 6144, "N": 32768, "n": 8, "x": "bf16",
         "out": "bf16", "pair": True, "act": "gelu", "tokens": 64, "gate": False, "spread": "even", "behind": 0},
        # Decode at the Grok-1 shape: down projection, rows scaled by their gates.
        {"name": "int8 down decode", "kind": "product", "R": 128, "K": 32768, "N": 6144, "n": 8, "x": "bf16",
         "out": "f32", "pair": False, "act": "gelu", "tokens": 0, "gate": True, "spread": "skewed", "behind": 0},
        # Prefill at the Grok-1 shape, T = 4096: gate and up projections.
        {"name": "int8 gate/up prefill", "kind": "product", "R": 8192, "K": 6144, "N": 32768, "n": 8, "x": "bf16",
         "out": "bf16", "pair": True, "act": "gelu", "tokens": 4096, "gate": False, "spread": "even", "behind": 0},
        # Prefill at the Grok-1 shape: down projection under skewed load.
        {"name": "int8 down prefill", "kind": "product", "R": 8192, "K": 32768, "N": 6144, "n": 8, "x": "bf16",
         "out": "f32", "pair": False, "act": "gelu", "tokens": 0, "gate": True, "spread": "skewed", "behind": 0},
        # One plain matrix of odd sizes on rows that are 8-bit already.
        {"name": "int8 plain odd", "kind": "product", "R": 333, "K": 1040, "N": 2064, "n": 1, "x": "i8",
         "out": "bf16", "pair": False, "act": "gelu", "tokens": 0, "gate": False, "spread": "even", "behind": 0},
        # Decode, T = 64: the two rows of each token.
        {"name": "combine decode", "kind": "combine", "T": 64, "k": 2, "d": 6144, "y": "f32", "out": "bf16",
         "weights": False, "residual": False, "missing": 0.0},
        # Prefill, T = 4096, eight rows of each token, weights and residual.
        {"name": "combine prefill", "kind": "combine", "T": 4096, "k": 8, "d": 6144, "y": "bf16", "out": "bf16",
         "weights": True, "residual": True, "missing": 0.0},
    ]


def spread_over(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "route", "route_grad", "product", "product", "product", "combine"])
    if kind in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * spread_over(rng, max(2, 8 // groups), 512 // groups)
        k = rng.randint(1, min(10, max(1, E // 2)))
        T = spread_over(rng, 1, 16384)
        T = max(1, min(T, 16384 * 256 // E))
        c = {"kind": kind, "T": T, "E": E, "k": k, "type": rng.choice(["f32", "bf16"]),
             "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.5,
             "scale": rng.choice([1.0, 2.5]), "valid": T if rng.random() < 0.6 else rng.randint(0, T),
             "mask": rng.choice([0.0, 0.0, 0.2])}
        if kind == "route":
            c.update({"groups": groups, "keep": rng.randint(1, groups), "rule": rng.choice(["max", "top2"]),
                      "bias": rng.random() < 0.5})
        else:
            c["scores"] = rng.random() < 0.5
        return c
    if kind == "combine":
        T, k, d = spread_over(rng, 1, 4096), rng.randint(1, 8), 8 * spread_over(rng, 8, 768)
        return {"kind": kind, "T": T, "k": k, "d": d, "y": rng.choice(["f32", "bf16"]),
                "out": rng.choice(["f32", "bf16"]), "weights": rng.random() < 0.5, "residual": rng.random() < 0.5,
                "missing": rng.choice([0.0, 0.1])}
    while True:
        pair = rng.random() < 0.5
        R, K, N = spread_over(rng, 1, 8192), 16 * spread_over(rng, 4, 2048), 16 * spread_over(rng, 4, 2048)
        n = rng.choice([1, 2, 8, 8, 16, 64])
        two = 2 if pair else 1
        if R * K * N * two <= 8192 * 6144 * 65536 and n * K * N * two <= 8 * 6144 * 65536 and R * N <= 8192 * 32768:
            break
    x = rng.choice(["bf16", "bf16", "f32", "i8"])
    return {"kind": kind, "R": R, "K": K, "N": N, "n": n, "x": x, "out": rng.choice(["bf16", "f32"]), "pair": pair,
            "act": rng.choice(["gelu", "gelu_erf", "silu"]),
            "tokens": spread_over(rng, 1, R) if x != "i8" and rng.random() < 0.5 else 0, "gate": rng.random() < 0.5,
            "spread": rng.choice(["even", "skewed", "holes"]), "behind": rng.choice([0, 0, R // 5])}


def rows_of(c):
    """Rows of each expert: shares by the case's spread, R - behind in all."""
    total, n = c["R"] - c["behind"], c["n"]
    share = {"even": np.ones(n), "skewed": 1.0 / np.arange(1, n + 1),
             "holes": (np.arange(n) % 3 != 1).astype(float)}[c["spread"]]
    edge = np.floor(np.cumsum(share) / share.sum() * total + 1e-9).astype(np.int64)
    edge[-1] = total
    return np.diff(np.concatenate([[0], edge]))


# ------------------------------------------------------------------ inputs --

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=DEV) * std

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    def int8(*shape):
        return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)

    def i32(*shape):
        return torch.zeros(shape, dtype=torch.int32, device=DEV)

    def f32(*shape):
        return torch.zeros(shape, device=DEV)

    s = {"case": c}
    if c["kind"] in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        l = normal(T, E)
        if c["mask"]:  # experts a token may not use, now and then all of them
            l[uniform(T, E) < c["mask"]] = -math.inf
            l[uniform(T) < 0.02] = -math.inf
        s["logits"] = l.to(TYPES[c["type"]])
        s["n_tokens"] = torch.full((1,), c["valid"], dtype=torch.int32, device=DEV)
        if c["kind"] == "route":
            s["bias"] = normal(E, std=0.05) if c["bias"] else None
            s["out"] = {"idx": i32(T, k), "weights": f32(T, k), "counts": i32(E), "offsets": i32(E + 1),
                        "perm_token": i32(T * k), "perm_slot": i32(T * k), "slot_pos": i32(T, k),
                        "gate_perm": f32(T * k)}
        else:
            idx = torch.argsort(uniform(T, E), dim=1)[:, :k].to(torch.int32)
            idx[torch.gather(s["logits"], 1, idx.long()) == -math.inf] = -1
            idx[c["valid"]:] = -1
            s["idx"] = idx.contiguous()
            s["grad_weights"] = normal(T, k)
            s["grad_scores"] = normal(T, E, std=0.1) if c["scores"] else None
            s["out"] = torch.zeros((T, E), dtype=TYPES[c["type"]], device=DEV)
    elif c["kind"] == "product":
        R, K, N, n = c["R"], c["K"], c["N"], c["n"]
        if c["x"] == "i8":
            s["x"] = int8(R, K)
            s["x_scale"] = uniform(R) * 0.02 + 0.005
        else:
            s["x"] = normal(c["tokens"] or R, K).to(TYPES[c["x"]])
            s["x_scale"] = None
        s["index"] = (torch.randint(0, c["tokens"], (R,), generator=g, device=DEV, dtype=torch.int32)
                      if c["tokens"] else None)
        s["counts"] = (None if n == 1 and c["behind"] == 0
                       else torch.tensor(rows_of(c), dtype=torch.int32, device=DEV))
        s["w"], s["w_up"] = int8(n, K, N), int8(n, K, N) if c["pair"] else None
        unit = 1.0 / (127 * math.sqrt(K))
        s["s"] = ((uniform(n, N) + 0.5) * unit).to(torch.bfloat16)
        s["s_up"] = ((uniform(n, N) + 0.5) * unit).to(torch.bfloat16) if c["pair"] else None
        s["gate"] = uniform(R) if c["gate"] else None
        s["out"] = torch.zeros((R, N), dtype=TYPES[c["out"]], device=DEV)
    else:
        T, k, d = c["T"], c["k"], c["d"]
        s["y"] = normal(T * k, d).to(TYPES[c["y"]])
        pos = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32).reshape(T, k)
        if c["missing"]:
            pos[uniform(T, k) < c["missing"]] = -1
        s["slot_pos"] = pos
        s["weights"] = uniform(T, k) if c["weights"] else None
        s["residual"] = normal(T, d).to(TYPES[c["out"]]) if c["residual"] else None
        s["out"] = torch.zeros((T, d), dtype=TYPES[c["out"]], device=DEV)
    return s


# -------------------------------------------------------------- plain form --

def plain_scores(l, c):
    """64-bit logits (NaN as -inf, +inf as the largest float) and their scores."""
    l = torch.where(torch.isnan(l), -math.inf, l.double()).clamp(max=FLT_MAX)
    ok = l > -math.inf
    if c["score"] == "sigmoid":
        return l, ok, torch.where(ok, 1 / (1 + torch.exp(-l)), 0.0)
    m = l.amax(1, keepdim=True)
    e = torch.where(ok, torch.exp(l - torch.where(m > -math.inf, m, 0.0)), 0.0)
    z = e.sum(1, keepdim=True)
    return l, ok, e / torch.where(z > 0, z, 1.0)


def plain_route(st):
    c = st["case"]
    T, E, k = c["T"], c["E"], c["k"]
    dev = st["logits"].device
    l, ok, s = plain_scores(st["logits"], c)
    ok = ok & (torch.arange(T, device=dev)[:, None] < st["n_tokens"])
    value = s if st["bias"] is None else s + st["bias"].double()
    rank = torch.where(ok, l if st["bias"] is None else value, -math.inf)
    if c["groups"] > 1:
        G = c["groups"]
        if c["rule"] == "max":
            gv = rank.view(T, G, -1).amax(2)
        else:
            two = torch.where(ok, value, -math.inf).view(T, G, -1).sort(dim=2, descending=True).values[:, :, :2]
            gv = torch.where(two[:, :, 0] > -math.inf, torch.where(two > -math.inf, two, 0.0).sum(2), -math.inf)
        first = gv.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=dev).scatter(1, first, True)
        rank = torch.where(kept.repeat_interleave(E // G, 1), rank, -math.inf)
    best, idx = rank.sort(dim=1, descending=True, stable=True)
    best, idx = best[:, :k], idx[:, :k]
    has = best > -math.inf
    w = torch.where(has, torch.gather(s, 1, idx), 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    w = (w * c["scale"]).float()
    idx = torch.where(has, idx, -1)
    e = idx.reshape(-1)
    key = torch.where(e < 0, E, e)
    order = key.sort(stable=True).indices
    counts = (key[:, None] == torch.arange(E, device=dev)).sum(0) if T * k * E < 1 << 20 else \
        torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    at = torch.arange(T * k, device=dev)
    used = at < offsets[E]
    pos = torch.empty_like(at)
    pos[order] = at
    return {"idx": idx.int(), "weights": w, "counts": counts.int(), "offsets": offsets.int(),
            "perm_token": torch.where(used, order // k, -1).int(), "perm_slot": torch.where(used, order % k, -1).int(),
            "slot_pos": torch.where(e < 0, -1, pos).int().view(T, k),
            "gate_perm": torch.where(used, w.reshape(-1)[order], 0.0)}


def plain_route_grad(st):
    c = st["case"]
    l, ok, s = plain_scores(st["logits"], c)
    row = torch.arange(c["T"], device=l.device)[:, None] < st["n_tokens"]
    s, has = s.float(), st["idx"] >= 0
    idx = torch.where(has, st["idx"], 0).long()
    g = torch.where(has, st["grad_weights"], 0.0) * c["scale"]
    if c["renorm"]:
        sel = torch.where(has, torch.gather(s, 1, idx), 0.0)
        total = sel.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        g = torch.where(has, (g - (g * sel / total).sum(1, keepdim=True)) / total, 0.0)
    ds = torch.zeros_like(s).scatter_add(1, idx, g)
    if st["grad_scores"] is not None:
        ds = ds + st["grad_scores"]
    dl = s * (1 - s) * ds if c["score"] == "sigmoid" else s * (ds - (ds * s).sum(1, keepdim=True))
    return torch.where(ok & row, dl, 0.0).to(st["logits"].dtype)


def plain_act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def plain_product(st):
    c = st["case"]
    x = st["x"] if st["index"] is None else st["x"][st["index"].long()]
    if c["x"] == "i8":
        q, a = x.float(), st["x_scale"]
    else:
        top = x.float().abs().amax(1, keepdim=True)
        # 64 bits: a quotient next to a half has to round the way the exact one does
        q = torch.round(x.double() * 127 / torch.where(top > 0, top, 1.0).double()).float()
        a = (top / 127)[:, 0]
    out = torch.zeros_like(st["out"])
    at = 0
    for e, m in enumerate(rows_of(c)):  # one product per expert with rows
        if m == 0:
            continue
        rows = slice(at, at + int(m))
        at += int(m)
        y = (q[rows] @ st["w"][e].float()) * a[rows, None] * st["s"][e].float()
        if c["pair"]:
            y = plain_act(y, c["act"]) * ((q[rows] @ st["w_up"][e].float()) * a[rows, None] * st["s_up"][e].float())
        out[rows] = (y if st["gate"] is None else y * st["gate"][rows, None]).to(out.dtype)
    return out


def plain_combine(st):
    pos = st["slot_pos"].long()
    rows = st["y"][pos.clamp(min=0)].float()
    w = (pos >= 0).float() if st["weights"] is None else torch.where(pos >= 0, st["weights"], 0.0)
    y = (rows * w[:, :, None]).sum(1)
    return (y if st["residual"] is None else y + st["residual"].float()).to(st["out"].dtype)


PLAIN = {"route": plain_route, "route_grad": plain_route_grad, "product": plain_product, "combine": plain_combine}


# --------------------------------------------------------------------- run --

def own_run(st):
    import mixture_experts_ffn_14_b200 as moe

    c = st["case"]
    if c["kind"] in ("route", "route_grad"):
        score = moe.MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else moe.MOE_SCORE_SOFTMAX
        if c["kind"] == "route":
            rule = moe.MOE_GROUP_TOP2_SUM if c["rule"] == "top2" else moe.MOE_GROUP_MAX
            return moe.moe_topk_route(st["logits"], c["k"], score=score, bias=st["bias"], n_groups=c["groups"],
                                      topk_groups=c["keep"], group_rule=rule, renormalize=c["renorm"],
                                      scale=c["scale"], n_tokens=st["n_tokens"], out=st["out"])
        return moe.moe_topk_route_backward(st["logits"], st["idx"], st["grad_weights"], score=score,
                                           renormalize=c["renorm"], scale=c["scale"], grad_scores=st["grad_scores"],
                                           n_tokens=st["n_tokens"], out=st["out"])
    if c["kind"] == "product":
        act = {"gelu": moe.MOE_ACT_GELU_TANH, "gelu_erf": moe.MOE_ACT_GELU_ERF, "silu": moe.MOE_ACT_SILU}[c["act"]]
        return moe.moe_int8_product(st["x"], st["w"], st["s"], x_scale=st["x_scale"], index=st["index"],
                                    counts=st["counts"], w_up=st["w_up"], s_up=st["s_up"], activation=act,
                                    gate=st["gate"], out=st["out"])
    return moe.moe_combine_topk(st["y"], st["slot_pos"], weights=st["weights"], residual=st["residual"],
                                out=st["out"])


def run(state):
    if own:
        return own_run(state)
    return PLAIN[state["case"]["kind"]](state)


def work(case):
    c = case
    if c["kind"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        out = T * k * (4 + 4) + T * k * (4 + 4 + 4 + 4) + E * 8
        return {"bytes": c["valid"] * E * BYTES[c["type"]] + out + (4 * E if c["bias"] else 0), "flops": 4 * T * E}
    if c["kind"] == "route_grad":
        T, E, k = c["T"], c["E"], c["k"]
        read = c["valid"] * (E * BYTES[c["type"]] + 8 * k + (4 * E if c["scores"] else 0))
        return {"bytes": read + T * E * BYTES[c["type"]], "flops": 6 * T * E}
    if c["kind"] == "product":
        K, N, two = c["K"], c["N"], 2 if c["pair"] else 1
        m = rows_of(c)
        rows = int(m.sum())
        weights = int((m > 0).sum()) * two * (K * N + 2 * N)
        return {"bytes": min(rows, c["tokens"] or rows) * K * BYTES[c["x"]] + weights + rows * N * BYTES[c["out"]],
                "flops": 2 * two * rows * K * N}
    T, k, d = c["T"], c["k"], c["d"]
    read = T * k * (d * BYTES[c["y"]] + 4) * (1 - c["missing"]) + (4 * T * k if c["weights"] else 0)
    return {"bytes": int(read) + T * d * BYTES[c["out"]] * (2 if c["residual"] else 1), "flops": 2 * T * k * d}


# ---------------------------------------------------- 64 bits, written apart --

def exact_scores(l, score):
    with np.errstate(over="ignore", invalid="ignore"):
        masked = ~(l > -np.inf)
        l = np.where(masked, -np.inf, np.minimum(l, FLT_MAX))
        if score == "sigmoid":
            p = np.where(l >= 0, 1 / (1 + np.exp(-np.abs(l))), np.exp(-np.abs(l)) / (1 + np.exp(-np.abs(l))))
        else:
            top = l.max(1)
            top[top == -np.inf] = 0
            p = np.exp(l - top[:, None])
            p /= np.maximum(p.sum(1), 1e-300)[:, None]
    p[masked] = 0
    return l, masked, p


def exact_route(c, st):
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    l, masked, p = exact_scores(st["logits"].double().cpu().numpy(), c["score"])
    masked[c["valid"]:] = True
    v = p + (0 if st["bias"] is None else st["bias"].double().cpu().numpy())
    r = np.where(masked, -np.inf, l if st["bias"] is None else v)
    if G > 1:
        v = np.where(masked, -np.inf, v if c["rule"] == "top2" else r).reshape(T, G, E // G)
        if c["rule"] == "top2":
            v = -np.sort(-v, axis=2)[:, :, :2]
            gv = np.where(np.isneginf(v[:, :, 0]), -np.inf, np.where(np.isneginf(v), 0, v).sum(2))
        else:
            gv = v.max(2)
        place = np.argsort(np.argsort(-gv, axis=1, kind="stable"), axis=1, kind="stable")
        r = np.where(np.repeat(place < c["keep"], E // G, axis=1), r, -np.inf)
    idx = np.argsort(-r, axis=1, kind="stable")[:, :k]
    idx[np.take_along_axis(r, idx, 1) == -np.inf] = -1
    w = np.where(idx < 0, 0, np.take_along_axis(p, np.maximum(idx, 0), 1))
    if c["renorm"]:
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    w = w * c["scale"]
    token, slot = np.nonzero(idx >= 0)
    order = np.lexsort((slot, token, idx[token, slot]))
    token, slot = token[order], slot[order]
    counts = np.array([(idx == e).sum() for e in range(E)]) if T * E < 1 << 16 else \
        np.bincount(idx[idx >= 0], minlength=E)
    n = len(token)
    out = {"idx": idx, "weights": w, "counts": counts, "offsets": np.concatenate([[0], np.cumsum(counts)]),
           "perm_token": np.full(T * k, -1), "perm_slot": np.full(T * k, -1), "slot_pos": np.full((T, k), -1),
           "gate_perm": np.zeros(T * k)}
    out["perm_token"][:n], out["perm_slot"][:n], out["gate_perm"][:n] = token, slot, w[token, slot]
    out["slot_pos"][token, slot] = np.arange(n)
    return {name: a if a.dtype == np.float64 else a.astype(np.int32) for name, a in out.items()}


def exact_route_grad(c, st):
    idx = st["idx"].cpu().numpy().astype(np.int64)
    l, masked, p = exact_scores(st["logits"].double().cpu().numpy(), c["score"])
    gw = st["grad_weights"].double().cpu().numpy() * c["scale"]
    rows = np.arange(c["T"])
    d = np.zeros_like(p) if st["grad_scores"] is None else st["grad_scores"].double().cpu().numpy()
    chosen = [np.where(idx[:, j] >= 0, p[rows, np.maximum(idx[:, j], 0)], 0) for j in range(c["k"])]
    total = np.maximum(sum(chosen), 1e-300)
    mean = sum(gw[:, j] * chosen[j] for j in range(c["k"])) / total
    for j in range(c["k"]):
        part = (gw[:, j] - mean) / total if c["renorm"] else gw[:, j]
        np.add.at(d, (rows, np.maximum(idx[:, j], 0)), np.where(idx[:, j] >= 0, part, 0))
    if c["score"] == "sigmoid":
        out = d * p * (1 - p)
    else:
        out = p * d - p * np.einsum("te,te->t", p, d)[:, None]
    out[masked] = 0
    out[c["valid"]:] = 0
    return out


def exact_act(z, act):
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu_erf":
        return z * torch.special.ndtr(z)
    return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))


def exact_product(c, st):
    x = st["x"].double()
    if st["index"] is not None:
        x = x.index_select(0, st["index"].long())
    if c["x"] == "i8":
        step = st["x_scale"].double()
    else:
        top = torch.linalg.vector_norm(x, float("inf"), dim=1)
        step = top / 127
        x = torch.round(127 * x / top.clamp(min=1e-300)[:, None])  # 127 x is exact: a half is met as one
    out = torch.zeros((c["R"], c["N"]), dtype=torch.float64, device=x.device)
    gate = torch.ones_like(step) if st["gate"] is None else st["gate"].double()
    ends = np.cumsum(rows_of(c))
    for e in range(c["n"]):
        a, b = int(ends[e - 1]) if e else 0, int(ends[e])
        if a < b:
            y = torch.mm(x[a:b] * step[a:b, None], st["w"][e].double() * st["s"][e].double())
            if c["pair"]:
                y = exact_act(y, c["act"]) * torch.mm(x[a:b] * step[a:b, None], st["w_up"][e].double()
                                                      * st["s_up"][e].double())
            out[a:b] = y * gate[a:b, None]
    return out


def exact_combine(c, st):
    out = torch.zeros((c["T"], c["d"]), dtype=torch.float64, device=st["y"].device)
    for j in range(c["k"]):
        pos = st["slot_pos"][:, j].long()
        part = st["y"][pos.clamp(min=0)].double()
        out += torch.where(pos[:, None] >= 0, part, 0.0) * (1.0 if st["weights"] is None
                                                            else st["weights"][:, j:j + 1].double())
    return out if st["residual"] is None else out + st["residual"].double()


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": exact_route, "route_grad": exact_route_grad, "product": exact_product,
            "combine": exact_combine}[case["kind"]](dict(case), st)
