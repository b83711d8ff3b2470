"""What the routing and 8-bit operators of the library are measured on.

Five operators that a mixture-of-experts layer needs beside the IQ_K experts:

* ``router_topk``       token -> (expert ids, weights) from the router's logits
* ``router_topk_grad``  the gradient of those weights with respect to the logits
* ``fp8_quantize``      activations to e4m3 with a float32 scale per 1 x 128 block
* ``fp8_linear``        activations times 8-bit weights with a scale per 128 x 128 block (the shared expert)
* ``moe_fp8``           the same product over expert-stacked weights at routed token-expert pairs

``run`` computes them in plain torch operations (``own`` false) or through the
library (``own`` true).  Sizes are those of the routed geometry the library is
built for (256 experts, top-6, hidden 4096, gate/up 2 x 2048) and generic ones.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0**-100
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def _blocks(n):
    return -(-n // BLOCK)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decoded token: latency; sigmoid scores, a balance bias, 8 groups of which 4 stay
        dict(name="router one token", op="router", T=1, E=256, k=6, scoring="sigmoid", bias=True, n_group=8,
             topk_group=4, group_top=2, renorm=True, scale=2.5, dtype="f32"),
        # a long batch of prompts: softmax of bf16 logits over the routed geometry
        dict(name="router 16384 tokens", op="router", T=16384, E=256, k=6, scoring="softmax", bias=False, n_group=1,
             topk_group=1, group_top=1, renorm=True, scale=1.0, dtype="bf16"),
        # a router being recalibrated on one 512-token sequence, weights not renormalised
        dict(name="router grad 512 tokens", op="router_grad", T=512, E=256, k=6, scoring="softmax", renorm=False,
             scale=1.0, dtype="f32"),
        # the same on a large odd batch with an expert count that is no power of two
        dict(name="router grad 8191 tokens", op="router_grad", T=8191, E=160, k=8, scoring="sigmoid", renorm=True,
             scale=2.5, dtype="bf16"),
        # activations of a few decoded tokens
        dict(name="quantize 8 tokens", op="quantize", M=8, K=4096, dtype="bf16"),
        # activations of a batch of prompts
        dict(name="quantize 8192 tokens", op="quantize", M=8192, K=4096, dtype="bf16"),
        # one decoded token through the shared expert's gate/up
        dict(name="linear 1 token", op="linear", M=1, N=4096, K=4096, dtype="bf16", out="f32"),
        # a ragged product: rows, columns and depth that fill no tile, the depth no whole block
        dict(name="linear 333 tokens ragged", op="linear", M=333, N=4001, K=2064, dtype="f32", out="bf16"),
        # a batch of prompts through the shared expert's gate/up
        dict(name="linear 8192 tokens", op="linear", M=8192, N=4096, K=4096, dtype="bf16", out="bf16"),
        # one decoded token at 6 of 256 experts, gate/up
        dict(name="experts 1 token", op="moe", T=1, k=6, E=256, N=4096, K=4096, slots=False, dtype="bf16",
             out="f32"),
        # a 512-token prompt at the down projection: each pair its own input, about 12 pairs per expert
        dict(name="experts 512 tokens", op="moe", T=512, k=6, E=256, N=4096, K=2048, slots=True, dtype="bf16",
             out="f32"),
        # a batch of prompts on one device's share of the experts, about 384 pairs per expert
        dict(name="experts 4096 tokens", op="moe", T=4096, k=6, E=64, N=2048, K=4096, slots=False, dtype="bf16",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(["router", "router_grad", "quantize", "linear", "linear", "moe", "moe"])
    if op in ("router", "router_grad"):
        E = rng.choice([8, 16, 60, 64, 96, 128, 160, 200, 256, 384, 512])
        k = rng.randint(1, min(10, E // 2))
        c = dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, scoring=rng.choice(["softmax", "sigmoid"]),
                 renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16", "f16"]))
        if op == "router":
            groups = rng.choice([g for g in (1, 2, 4, 8) if E % g == 0 and E // g >= 2])
            keep = groups if groups == 1 else rng.randint(1, groups)
            while keep * (E // groups) < k:
                keep += 1
            c.update(bias=rng.random() < 0.5, n_group=groups, topk_group=keep, group_top=rng.choice([1, 2]))
        return c
    if op == "quantize":
        return dict(op=op, M=_log(rng, 1, 8192), K=16 * _log(rng, 8, 512), dtype=rng.choice(["f32", "bf16", "f16"]))
    if op == "linear":
        return dict(op=op, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192), K=16 * _log(rng, 16, 512),
                    dtype=rng.choice(["f32", "bf16", "f16"]), out=rng.choice(["f32", "bf16", "f16"]))
    E = rng.choice([8, 16, 60, 64, 128, 256])
    return dict(op=op, T=_log(rng, 1, 4096), k=rng.randint(1, min(8, E // 2)), E=E, N=_log(rng, 128, 4096),
                K=16 * _log(rng, 16, 256), slots=rng.random() < 0.4, dtype=rng.choice(["f32", "bf16"]),
                out=rng.choice(["f32", "f32", "bf16", "f16"]))


def draw(rng):
    """One more case of the same ranges, at most as much work as the largest listed case of its operator."""
    while True:
        c = _draw(rng)
        if c["op"] == "linear" and c["N"] == 3072 or c["op"] == "moe" and c["N"] == 3072 or c.get("K") == 3072:
            continue
        most = [work(x) for x in listed() if x["op"] == c["op"]]
        w = work(c)
        if all(w[m] <= max(x[m] for x in most) for m in ("bytes", "flops")):
            return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _logits(case, gen):
    """Router logits: a spread per token on top of each expert's own level."""
    T, E = case["T"], case["E"]
    base = torch.randn(E, generator=gen, device="cuda") * 0.5
    return ((torch.randn(T, E, generator=gen, device="cuda") * 1.5 + base)).to(TYPES[case["dtype"]])


def _hangs(case, logits, bias):
    """Rows whose choice hangs on the last bits: two values that decide it differ, but by less than float32
    arithmetic resolves.  (Equal values are no such case: the lowest index wins.)"""
    l = logits.double()
    T, E = l.shape
    s = torch.sigmoid(l) if case["scoring"] == "sigmoid" else torch.softmax(l, -1)
    c = l if bias is None else s + bias.double()

    def near(v, n):
        v = v.sort(dim=-1, descending=True).values[:, : n + 1]
        gap = v[:, :-1] - v[:, 1:]
        return ((gap > 0) & (gap < 4e-6 * v[:, :-1].abs().clamp_min(1e-30))).any(-1)

    bad = torch.zeros(T, dtype=torch.bool, device=l.device)
    G = case["n_group"]
    if G > 1:
        two = case["group_top"] == 2 and E // G > 1
        g = (s if bias is None and two else c).view(T, G, E // G).topk(2 if two else 1, -1).values.sum(-1)
        if bias is not None or two:
            bad |= near(g, G - 1)
        g = g.sort(dim=-1, descending=True, stable=True).indices[:, : case["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, g, True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, c.new_full((), -math.inf))
    if bias is not None:
        bad |= near(torch.where(torch.isinf(c), c.new_full((), -1e30), c), min(case["k"], E - 1))
    return bad


def _weights(E, N, K, gen):
    """8-bit expert weights with a scale per 128 x 128 block: codes [E, N, K], scales [E, N / 128, K / 128]."""
    nb, kb = _blocks(N), _blocks(K)
    codes = torch.empty(E, N, K, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(E, nb, kb, device="cuda")
    step = max(1, (1 << 28) // (N * K))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn(n, N, K, generator=gen, device="cuda")
        level = torch.rand(n, nb, kb, generator=gen, device="cuda") + 0.5
        a = 4.5 * level / math.sqrt(K)  # a block's largest weight, about
        scales[e : e + n] = a / E4M3_MAX
        codes[e : e + n] = (w * (E4M3_MAX / 4.5)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, scales


def _activations(rows, K, dtype, gen):
    """Activations as they come out of a norm: unit spread, a few channels far larger than the others."""
    x = torch.randn(rows, K, generator=gen, device="cuda")
    loud = torch.rand(K, generator=gen, device="cuda") < 0.005
    return (x * torch.where(loud, 20.0, 1.0)).to(TYPES[dtype])


def _ids(T, k, E, gen):
    """k different experts for each token, some experts taken more often than others."""
    level = torch.randn(E, generator=gen, device="cuda") * 0.3
    noise = -torch.log(-torch.log(torch.rand(T, E, generator=gen, device="cuda").clamp(1e-6, 1 - 1e-6)))
    return (noise + level).topk(k, -1).indices.to(torch.int32).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    state = {"case": case}
    op = case["op"]
    if op == "router":
        bias = None
        if case["bias"]:  # a balance bias that is moved in steps of 0.001
            bias = torch.randint(-100, 101, (case["E"],), generator=gen, device="cuda").float() * 0.001
        logits = _logits(case, gen)
        for _ in range(20):
            bad = _hangs(case, logits, bias)
            if not bool(bad.any()):
                break
            logits = torch.where(bad[:, None], _logits(case, gen), logits)
        state.update(logits=logits, bias=bias)
    elif op == "router_grad":
        logits = _logits(case, gen)
        ids = logits.float().sort(dim=-1, descending=True, stable=True).indices[:, : case["k"]].to(torch.int32).contiguous()
        state.update(logits=logits, ids=ids, dw=torch.randn(case["T"], case["k"], generator=gen, device="cuda"))
    elif op == "quantize":
        state.update(x=_activations(case["M"], case["K"], case["dtype"], gen))
    elif op == "linear":
        codes, scales = _weights(1, case["N"], case["K"], gen)
        state.update(codes=codes, scales=scales, x=_activations(case["M"], case["K"], case["dtype"], gen))
    else:
        codes, scales = _weights(case["E"], case["N"], case["K"], gen)
        slots = case["k"] if case["slots"] else 1
        state.update(codes=codes, scales=scales, slots=slots, ids=_ids(case["T"], case["k"], case["E"], gen),
                     x=_activations(case["T"] * slots, case["K"], case["dtype"], gen))
    return state


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------


def _plain_router(logits, bias, case):
    l = logits.float()
    T, E = l.shape
    if case["scoring"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        s = torch.exp(l - l.max(-1, keepdim=True).values)
        s = s / s.sum(-1, keepdim=True)
    c = l if bias is None else s + bias
    G = case["n_group"]
    if G > 1:
        if case["group_top"] == 2:
            g = (s if bias is None else c).view(T, G, E // G)
            g = g.sort(dim=-1, descending=True).values[..., :2].sum(-1)
        else:
            g = c.view(T, G, E // G).max(-1).values
        g = g.sort(dim=-1, descending=True, stable=True).indices[:, : case["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device).scatter_(1, g, True)
        c = torch.where(keep.repeat_interleave(E // G, 1), c, -math.inf)
    ids = c.sort(dim=-1, descending=True, stable=True).indices[:, : case["k"]]
    w = s.gather(1, ids)
    if case["renorm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": w * case["scale"]}


def _plain_router_grad(logits, ids, dw, case):
    l = logits.float()
    if case["scoring"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
    else:
        s = torch.exp(l - l.max(-1, keepdim=True).values)
        s = s / s.sum(-1, keepdim=True)
    ids = ids.long()
    chosen = s.gather(1, ids)
    g = dw * case["scale"]
    if case["renorm"]:
        d = chosen.sum(-1, keepdim=True)
        g = (g - (g * chosen).sum(-1, keepdim=True) / d) / d
    ds = torch.zeros_like(l).scatter_(1, ids, g)
    if case["scoring"] == "sigmoid":
        dl = ds * s * (1.0 - s)
    else:
        dl = s * (ds - (ds * s).sum(-1, keepdim=True))
    return dl.to(logits.dtype)


def _plain_quantize(x):
    M, K = x.shape
    kb = _blocks(K)
    v = torch.nn.functional.pad(x.float(), (0, kb * BLOCK - K)).view(M, kb, BLOCK)
    a = v.abs().amax(-1).clamp_min(AMAX_FLOOR)
    q = (v * torch.div(torch.full_like(a, E4M3_MAX), a)[..., None]).to(torch.float8_e4m3fn)
    return q.view(M, kb * BLOCK)[:, :K].contiguous(), a / E4M3_MAX


def _widen(codes, scales):
    """The float32 values that e4m3 codes [E, N, K] (or [M, K]) stand for."""
    *_, N, K = codes.shape
    s = scales.repeat_interleave(BLOCK, -1)[..., :K]
    if codes.dim() == 3:
        s = s.repeat_interleave(BLOCK, -2)[..., :N, :]
    return codes.float() * s


def _plain_linear(codes, scales, x, out):
    q, s = _plain_quantize(x)
    return (_widen(q, s) @ _widen(codes, scales)[0].t()).to(TYPES[out])


def _plain_moe(codes, scales, x, ids, slots, out):
    T, k = ids.shape
    N, K = codes.shape[1:]
    q, s = _plain_quantize(x)
    xq = _widen(q, s)
    # the experts in use, each with its pairs in a padded buffer
    used, at, counts = torch.unique(ids.reshape(-1).long(), return_inverse=True, return_counts=True)
    order = at.argsort(stable=True)
    rank = torch.arange(T * k, device=x.device) - (counts.cumsum(0) - counts)[at[order]]
    most = int(counts.max())
    rows = order // k if slots == 1 else order
    buf = torch.zeros(len(used), most, K, device=x.device)
    buf[at[order], rank] = xq[rows]
    w = _widen(codes.view(torch.uint8)[used].view(torch.float8_e4m3fn), scales[used])
    y = torch.bmm(w, buf.transpose(1, 2).contiguous())
    res = torch.empty(T * k, N, device=x.device)
    res[order] = y.transpose(1, 2)[at[order], rank]
    return res.view(T, k, N).to(TYPES[out])


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import dequant_iqk_moe_amd as q

        if op == "router":
            ids, w = q.router_topk(state["logits"], case["k"], scoring=case["scoring"], bias=state["bias"],
                                   n_group=case["n_group"], topk_group=case["topk_group"],
                                   group_top=case["group_top"], renorm=case["renorm"], scale=case["scale"])
            return {"ids": ids, "weights": w}
        if op == "router_grad":
            return {"dlogits": q.router_topk_grad(state["logits"], state["ids"], state["dw"], scoring=case["scoring"],
                                                  renorm=case["renorm"], scale=case["scale"])}
        if op == "quantize":
            codes, scales = q.fp8_quantize(state["x"])
            return {"codes": codes, "scales": scales}
        w = q.Fp8Weights(state["codes"], state["scales"])
        if op == "linear":
            return {"y": q.fp8_linear(w, state["x"], out_dtype=TYPES[case["out"]])}
        return {"y": q.moe_fp8(w, state["x"], state["ids"], x_slots=state["slots"],
                               out_dtype=TYPES[case["out"]])}
    if op == "router":
        return _plain_router(state["logits"], state["bias"], case)
    if op == "router_grad":
        return {"dlogits": _plain_router_grad(state["logits"], state["ids"], state["dw"], case)}
    if op == "quantize":
        codes, scales = _plain_quantize(state["x"])
        return {"codes": codes, "scales": scales}
    if op == "linear":
        return {"y": _plain_linear(state["codes"], state["scales"], state["x"], case["out"])}
    return {"y": _plain_moe(state["codes"], state["scales"], state["x"], state["ids"], state["slots"], case["out"])}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "router":
        T, E, k = case["T"], case["E"], case["k"]
        b = T * E * BYTES[case["dtype"]] + T * k * 8 + (E * 4 if case["bias"] else 0)
        return {"bytes": b, "flops": T * E * 4}
    if op == "router_grad":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": 2 * T * E * BYTES[case["dtype"]] + T * k * 8, "flops": T * E * 6}
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (BYTES[case["dtype"]] + 1) + M * _blocks(K) * 4, "flops": 2 * M * K}
    N, K = case["N"], case["K"]
    expert = N * K + _blocks(N) * _blocks(K) * 4
    if op == "linear":
        M = case["M"]
        return {"bytes": expert + M * K * BYTES[case["dtype"]] + M * N * BYTES[case["out"]], "flops": 2 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    P = T * k
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token takes, about
    b = used * expert + T * (k if case["slots"] else 1) * K * BYTES[case["dtype"]] + P * 4 + P * N * BYTES[case["out"]]
    return {"bytes": b, "flops": 2 * P * N * K}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_codes(x):
    """The quantisation's definition: the float32 reciprocal and product are part of it and are rounded here from
    64-bit values; the rounding to e4m3 (to nearest, ties to even) is taken on the grid of its values."""
    x = x.double()
    M, K = x.shape
    kb = _blocks(K)
    codes = torch.zeros_like(x)
    scales = torch.empty(M, kb, dtype=torch.float64, device=x.device)
    for b in range(kb):
        v = x[:, b * BLOCK : (b + 1) * BLOCK]
        a = torch.maximum(v.abs().amax(1), torch.full_like(v[:, 0], AMAX_FLOOR))
        r = (E4M3_MAX / a).float().double()
        v = (v * r[:, None]).float().double()
        e = torch.floor(torch.log2(v.abs().clamp_min(2.0**-40))).clamp(min=-6.0)
        grid = torch.exp2(e - 3.0)
        codes[:, b * BLOCK : (b + 1) * BLOCK] = torch.round(v / grid) * grid
        scales[:, b] = a / E4M3_MAX
    return codes, scales


def _exact_scaled(codes, scales):
    out = codes.double()
    for b in range(scales.shape[-1]):
        part = out[..., b * BLOCK : (b + 1) * BLOCK]
        if codes.dim() == 2 and scales.shape[0] == codes.shape[0]:  # a scale per row and block
            part *= scales[:, b : b + 1]
        else:  # a scale per 128 rows and block
            rows = torch.arange(codes.shape[0], device=codes.device) // BLOCK
            part *= scales[rows, b].double()[:, None]
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("router", "router_grad"):
        l = state["logits"].double()
        T, E = l.shape
        s = torch.sigmoid(l) if case["scoring"] == "sigmoid" else torch.softmax(l, 1)
        if op == "router":
            c = l if state["bias"] is None else s + state["bias"].double()
            score = s if state["bias"] is None else c
            G = case["n_group"]
            per = E // G
            best = []
            for g in range(G):
                part = score if case["group_top"] == 2 else c
                best.append(part[:, g * per : (g + 1) * per].topk(case["group_top"], 1).values.sum(1))
            best = torch.stack(best, 1)
            order = torch.argsort(-best, dim=1, stable=True)
            for g in range(G):
                gone = (order[:, case["topk_group"] :] == g).any(1)
                c = c.clone()
                c[gone, g * per : (g + 1) * per] = -math.inf
            ids = torch.argsort(-c, dim=1, stable=True)[:, : case["k"]]
            w = torch.gather(s, 1, ids)
            if case["renorm"]:
                w = w / w.sum(1, keepdim=True)
            return {"ids": ids.to(torch.int32), "weights": w * case["scale"]}
        ids = state["ids"].long()
        z = torch.zeros_like(l, requires_grad=True)
        with torch.enable_grad():
            v = l + z
            p = torch.sigmoid(v) if case["scoring"] == "sigmoid" else torch.softmax(v, 1)
            w = torch.gather(p, 1, ids)
            if case["renorm"]:
                w = w / w.sum(1, keepdim=True)
            (w * case["scale"] * state["dw"].double()).sum().backward()
        return {"dlogits": z.grad}
    codes, scales = _exact_codes(state["x"])
    if op == "quantize":
        return {"codes": codes, "scales": scales}
    x = _exact_scaled(codes, scales)
    if op == "linear":
        w = state["codes"][0].double()
        for n in range(0, case["N"], BLOCK):
            for b in range(_blocks(case["K"])):
                w[n : n + BLOCK, b * BLOCK : (b + 1) * BLOCK] *= state["scales"][0, n // BLOCK, b].double()
        return {"y": x @ w.t()}
    ids = state["ids"]
    T, k = ids.shape
    y = torch.empty(T, k, case["N"], dtype=torch.float64, device=x.device)
    for e in range(case["E"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            rows = t if state["slots"] == 1 else t * k + j
            blocks = state["scales"][e].double()
            grown = blocks[:, None, :, None].expand(-1, BLOCK, -1, BLOCK).reshape(
                blocks.shape[0] * BLOCK, blocks.shape[1] * BLOCK)[: case["N"], : case["K"]]
            y[t, j] = x[rows] @ (state["codes"][e].double() * grown).t()
    return {"y": y}
