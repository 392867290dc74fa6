"""Operators of a mixture-of-experts layer around token dispatch and combine,
as cases to be timed and compared.

Three operators and their directions:

* the router: scores of each token's logits (softmax or sigmoid), the choice
  of k experts (with a selection bias and expert groups), their weights, and
  the gradient back to the logits;
* token rows sorted by expert and back, in any of bf16 / fp16 / fp32, any
  width and row stride, with weights applied on either way, and the gradients;
* the experts' products with 4-bit weights and group scales for few rows per
  expert (a plain matrix-vector product where there is one expert), rows
  gathered from the tokens, optionally with the gated activation.

``run`` computes them in plain torch operations when ``own`` is false and
through this repository's entry points when it is true.  ``exact`` is a
second, independent computation in 64 bits.
"""

import math

import torch

own = False

DEV = "cuda:0"
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------- the cases --

def _router(name, kind, T, E, k, dtype, score, bias=False, groups=1, topk_groups=1, group_top=1,
            renorm=True, scale=1.0, probs=False, masked=0.0, pad=0):
    return dict(name=name, kind=kind, T=T, E=E, k=k, dtype=dtype, score=score, bias=bias,
                groups=groups, topk_groups=topk_groups, group_top=group_top, renorm=renorm,
                scale=scale, probs=probs, masked=masked, pad=pad)


def _rows(name, kind, T, H, E, k, dtype, weighted=True, masked=0.0, pad=0):
    return dict(name=name, kind=kind, T=T, H=H, E=E, k=k, dtype=dtype, weighted=weighted,
                masked=masked, pad=pad)


def _w4(name, T, E, k, K, N, group, dtype, zeros=False, glu=False, gather=True):
    return dict(name=name, kind="w4", T=T, E=E, k=k, K=K, N=N, group=group, dtype=dtype,
                zeros=zeros, glu=glu, gather=gather)


def listed():
    return [
        # one decoded token choosing 8 of 256 experts through 4 of 8 groups
        # with a selection bias: nothing but latency
        _router("router_1_token", "router", 1, 256, 8, "bf16", "sigmoid", bias=True, groups=8,
                topk_groups=4, group_top=2, scale=2.5),
        # a training step of 8192 tokens over 256 experts, all probabilities
        # returned for a load-balancing loss
        _router("router_8192_probs", "router", 8192, 256, 8, "fp32", "softmax", probs=True),
        # its gradient, from the weights' and the probabilities' gradients
        _router("router_8192_backward", "router_bwd", 8192, 256, 8, "fp32", "softmax", probs=True),
        # an odd batch over 60 experts, logits inside a wider buffer, some
        # experts masked for some tokens and a few tokens with none left
        _router("router_ragged", "router", 1021, 60, 4, "fp16", "sigmoid", bias=True,
                masked=0.2, renorm=False, pad=5),
        # fp16 rows of a mid-size layer, weights applied on the way in
        _rows("permute_fp16", "permute", 4096, 2048, 64, 4, "fp16"),
        # fp32 rows of odd width inside a wider buffer, 5% of the choices masked
        _rows("unpermute_odd_fp32", "unpermute", 1021, 1999, 64, 4, "fp32", masked=0.05, pad=3),
        # the gradient of the weighted permute at the largest size, bf16
        _rows("permute_backward_8192", "permute_bwd", 8192, 7168, 256, 8, "bf16"),
        # the gradient of the weighted sum of expert outputs, fp16
        _rows("unpermute_backward_fp16", "unpermute_bwd", 4096, 2048, 64, 4, "fp16"),
        # one token through the gated first product of its 8 experts (of 256)
        _w4("w4_1_token_gated", 1, 256, 8, 7168, 4096, 128, "bf16", glu=True),
        # 64 tokens through the second product: most experts hold 1 to 5 rows
        _w4("w4_64_tokens", 64, 256, 8, 2048, 7168, 128, "bf16", gather=False),
        # a few tokens, fine groups with zero points, odd output width, fp16
        _w4("w4_3_tokens_zeros", 3, 64, 4, 2048, 1411, 32, "fp16", zeros=True),
        # a short prompt of 512 tokens: about 64 rows per expert
        _w4("w4_512_tokens_gated", 512, 64, 8, 2048, 2816, 128, "bf16", glu=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["router", "router_bwd", "permute", "permute_bwd", "unpermute",
                       "unpermute_bwd", "w4", "w4"])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    if kind.startswith("router"):
        E = rng.choice([8, 16, 60, 64, 96, 128, 160, 256])
        groups = rng.choice([1, 1, 2, 4]) if E % 4 == 0 else 1
        c = _router("", kind, _log(rng, 1, 8192), E, rng.randint(1, 8), dtype,
                    rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    topk_groups=max(1, groups // 2), group_top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                    probs=rng.random() < 0.5, masked=rng.choice([0.0, 0.1]), pad=rng.choice([0, 0, 3]))
        c["k"] = min(c["k"], E // groups * c["topk_groups"])
    elif kind == "w4":
        E = rng.choice([1, 8, 16, 64, 128])
        glu = rng.random() < 0.5
        K = 32 * _log(rng, 8, 160)
        N = _log(rng, 96, 4096)
        N += N % 2 if glu else 0
        c = _w4("", _log(rng, 1, 512), E, rng.randint(1, min(8, E)), K, N,
                rng.choice([32, 64, 128, 128]), rng.choice(["bf16", "fp16"]),
                zeros=rng.random() < 0.5, glu=glu, gather=rng.random() < 0.5)
        while c["E"] * c["N"] * c["K"] > 5e8:
            c["N"] = max(96, c["N"] // 4 * 2)
            c["E"] = max(8, c["E"] // 2)
            c["k"] = min(c["k"], c["E"])
    else:
        E = rng.choice([8, 16, 64, 160, 256])
        k = rng.randint(1, 8)
        H = _log(rng, 64, 7168)
        T = _log(rng, 1, 8192)
        while T * k * H * _BYTES[dtype] > 4e8:
            T = max(1, T * 2 // 3)
        c = _rows("", kind, T, H, E, k, dtype, weighted=rng.random() < 0.75,
                  masked=rng.choice([0.0, 0.05]), pad=rng.choice([0, 0, 1, 8]))
    c.pop("name")
    return c


# ---------------------------------------------------------------- the inputs --

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _wide(T, H, pad, dtype, g):
    """[T, H] normal values, inside a buffer of H + pad columns."""
    return torch.randn(T, H + pad, generator=g, device=DEV).to(dtype)[:, :H]


def _routing(T, E, k, masked, g):
    """k distinct experts per token in random order, a fraction masked."""
    idx = torch.rand(T, E, generator=g, device=DEV).argsort(1)[:, :k].contiguous()
    if masked:
        idx[torch.rand(T, k, generator=g, device=DEV) < masked] = -1
    return idx


def _layout(idx, E):
    """Stable sort of the choices by expert: the layout a program has in hand
    once it has chosen (counts, offsets, slot [T, k], source token per row)."""
    T, k = idx.shape
    flat = idx.reshape(-1)
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = torch.sort(key, stable=True).indices
    slot = torch.empty_like(flat)
    slot[order] = torch.arange(T * k, device=DEV)
    slot = torch.where(flat < 0, torch.full_like(slot, -1), slot)
    counts = (key[:, None] == torch.arange(E, device=DEV)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return (counts.int(), offsets.int(), slot.int().reshape(T, k), (order // k).int())


def prepare(case, seed):
    c, g = case, _gen(seed)
    dt = _TYPES[c["dtype"]]
    s = dict(case=c)
    if c["kind"] in ("router", "router_bwd"):
        T, E, k = c["T"], c["E"], c["k"]
        buf = torch.randn(T, E + c["pad"], generator=g, device=DEV) * 1.5
        if c["masked"]:
            buf[torch.rand(T, E + c["pad"], generator=g, device=DEV) < c["masked"]] = -math.inf
            buf[torch.rand(T, generator=g, device=DEV) < 0.01] = -math.inf
        s["logits"] = buf.to(dt)[:, :E]
        s["bias"] = (torch.rand(E, generator=g, device=DEV) * 0.2 - 0.1) if c["bias"] else None
        if c["kind"] == "router_bwd":
            s["topk_idx"] = _choose(s["logits"], s["bias"], c)
            s["grad_weights"] = torch.randn(T, k, generator=g, device=DEV)
            s["grad_probs"] = torch.randn(T, E, generator=g, device=DEV) if c["probs"] else None
        return s
    if c["kind"] == "w4":
        T, E, k, K, N, G = c["T"], c["E"], c["k"], c["K"], c["N"], c["group"]
        idx = _routing(T, E, k, 0.0, g)
        _, s["offsets"], _, src = _layout(idx, E)
        s["src"] = src if c["gather"] else None
        s["x"] = torch.randn(T if c["gather"] else T * k, K, generator=g, device=DEV).to(dt)
        ng = (K + G - 1) // G
        codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
        scales = ((torch.rand(E, N, ng, generator=g, device=DEV) + 0.5) / (4.6 * math.sqrt(K))).to(dt)
        zeros = torch.randint(5, 12, (E, N, ng), generator=g, device=DEV, dtype=torch.uint8) if c["zeros"] else None
        s["rows"] = T * k
        if own:   # the weights are laid out once, when a program loads them
            from combine_ep_layout_04_amd import ep
            s["weights"] = ep.ep_w4_pack(codes, scales, zeros, group_size=G, gated=c["glu"])
        else:     # and the plain program keeps them, and its segment bounds, as they are
            s["codes"], s["scales"], s["zeros"] = codes, scales, zeros
            s["bounds"] = s["offsets"].tolist()
        return s
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    idx = _routing(T, E, k, c["masked"], g) if k <= E else torch.randint(0, E, (T, k), generator=g, device=DEV)
    s["counts"], s["offsets"], s["slot"], _ = _layout(idx, E)
    w = torch.rand(T, k, generator=g, device=DEV)
    s["weights"] = w / w.sum(1, keepdim=True) if c["weighted"] else None
    s["rows"] = R = T * k
    if c["kind"] in ("permute", "permute_bwd", "unpermute_bwd"):
        s["x"] = _wide(T, H, c["pad"], dt, g)      # tokens, or the gradient of the sum
    if c["kind"] in ("unpermute", "permute_bwd", "unpermute_bwd"):
        s["y"] = _wide(R, H, c["pad"], dt, g)      # rows by expert, or their gradient
    return s


# -------------------------------------------------------------- plain forms --

def _choose(logits, bias, c):
    """The k chosen experts per token in 64 bits, best first, ties to the
    lowest index; -1 where fewer than k are left."""
    T, E, k = c["T"], c["E"], c["k"]
    l = logits.double()
    none = l == -math.inf
    if c["score"] == "softmax":
        m = l.max(1, keepdim=True).values
        p = torch.where(none, 0.0, torch.exp(l - m))
        score = p / p.sum(1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-l))
    val = score + bias.double() if bias is not None else score
    order = val if bias is not None else l
    order = torch.where(none, -math.inf, order)
    if c["groups"] > 1:
        n = c["groups"]
        # a group is as good as its best logit, or its best scores added up
        by = val if bias is not None or c["group_top"] > 1 else l
        by = torch.where(none, -math.inf, by).reshape(T, n, E // n)
        top = by.sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        some = (top[:, :, :1] != -math.inf).squeeze(2)
        gs = torch.where(some, torch.where(top == -math.inf, 0.0, top).sum(2), -math.inf)
        best = gs.sort(dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros(T, n, dtype=torch.bool, device=DEV).scatter_(1, best, True)
        order = torch.where(keep.repeat_interleave(E // n, 1), order, -math.inf)
    v, i = order.sort(dim=1, descending=True, stable=True)
    return torch.where(v[:, :k] == -math.inf, -1, i[:, :k])


def _router_parts(logits, idx, c):
    """Probabilities of all experts and weights of the chosen ones, fp32."""
    l = logits.float()
    if c["score"] == "softmax":
        m = l.max(1, keepdim=True).values
        e = torch.exp(l - torch.where(m == -math.inf, 0.0, m))
        z = e.sum(1, keepdim=True)
        p = e / torch.where(z == 0, 1.0, z)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    sel = torch.where(idx < 0, 0.0, p.gather(1, idx.clamp(min=0)))
    if c["renorm"]:
        d = sel.sum(1, keepdim=True)
        sel = sel / torch.where(d == 0, 1.0, d)
    return p, sel * c["scale"]


def _plain_router(s):
    c = s["case"]
    idx = _choose(s["logits"], s["bias"], c)
    p, w = _router_parts(s["logits"], idx, c)
    return (idx, w, p) if c["probs"] else (idx, w)


def _plain_router_bwd(s):
    c, idx, gw = s["case"], s["topk_idx"], s["grad_weights"]
    p, w = _router_parts(s["logits"], idx, c)
    r = w / c["scale"]
    at = idx.clamp(min=0)
    gsel = gw * c["scale"]
    if c["renorm"]:
        sel = torch.where(idx < 0, 0.0, p.gather(1, at))
        d = sel.sum(1, keepdim=True)
        gsel = (gsel - (gsel * r).sum(1, keepdim=True)) / torch.where(d == 0, 1.0, d)
    gsel = torch.where(idx < 0, 0.0, gsel)
    gp = torch.zeros_like(p) if s["grad_probs"] is None else s["grad_probs"].clone()
    gp.scatter_add_(1, at, gsel)
    if c["score"] == "softmax":
        gl = p * (gp - (p * gp).sum(1, keepdim=True))
    else:
        gl = gp * p * (1.0 - p)
    return gl.to(s["logits"].dtype)


def _plain_rows(s):
    c, kind, slot = s["case"], s["case"]["kind"], s["slot"].long()
    T, H, k, R = c["T"], c["H"], c["k"], s["rows"]
    dt = _TYPES[c["dtype"]]
    ok = slot >= 0
    at = slot.clamp(min=0)
    w = s["weights"] if s["weights"] is not None else torch.ones(T, k, device=DEV)
    if kind in ("permute", "unpermute_bwd"):
        x = s["x"].float()
        rows = torch.zeros(R + 1, H, dtype=dt, device=DEV)
        gw = torch.zeros(T, k, device=DEV)
        for j in range(k):
            # a masked choice goes to the row past the end
            rows[torch.where(ok[:, j], at[:, j], R)] = (x * w[:, j, None]).to(dt)
            if kind == "unpermute_bwd" and s["weights"] is not None:
                gw[:, j] = torch.where(ok[:, j], (x * s["y"][at[:, j]].float()).sum(1), 0.0)
        rows = rows[:R]
        if kind == "permute" or s["weights"] is None:
            return rows
        return rows, gw
    out = torch.zeros(T, H, device=DEV)
    gw = torch.zeros(T, k, device=DEV)
    for j in range(k):
        row = s["y"][at[:, j]].float()
        out += torch.where(ok[:, j, None], w[:, j, None] * row, 0.0)
        if kind == "permute_bwd" and s["weights"] is not None:
            gw[:, j] = torch.where(ok[:, j], (s["x"].float() * row).sum(1), 0.0)
    out = out.to(dt)
    return (out, gw) if kind == "permute_bwd" and s["weights"] is not None else out


def _plain_w4(s):
    c = s["case"]
    K, N, G = c["K"], c["N"], c["group"]
    x = s["x"] if s["src"] is None else s["x"][s["src"].long()]
    x = x.float()
    out = torch.empty(s["rows"], N, device=DEV)
    for e in range(c["E"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if a == b:
            continue
        q = torch.stack([s["codes"][e] & 15, s["codes"][e] >> 4], 2).reshape(N, K).float()
        z = 8.0 if s["zeros"] is None else s["zeros"][e].float().repeat_interleave(G, 1)[:, :K]
        w = (q - z) * s["scales"][e].float().repeat_interleave(G, 1)[:, :K]
        out[a:b] = x[a:b] @ w.t()
    if c["glu"]:
        gate, up = out[:, :N // 2], out[:, N // 2:]
        out = gate / (1.0 + torch.exp(-gate)) * up
    return out.to(s["x"].dtype)


# ------------------------------------------------------------------ one pass --

def run(state):
    s = state
    c = s["case"]
    kind = c["kind"]
    if not own:
        return {"router": _plain_router, "router_bwd": _plain_router_bwd,
                "w4": _plain_w4}.get(kind, _plain_rows)(s)
    from combine_ep_layout_04_amd import ep
    if kind == "router":
        idx, w, p = ep.ep_router(s["logits"], c["k"], score=c["score"], bias=s["bias"],
                                 num_groups=c["groups"], topk_groups=c["topk_groups"],
                                 group_top=c["group_top"], renormalize=c["renorm"],
                                 scale=c["scale"], want_probs=c["probs"])
        return (idx, w, p) if c["probs"] else (idx, w)
    if kind == "router_bwd":
        return ep.ep_router_backward(s["logits"], s["topk_idx"], s["grad_weights"],
                                     s["grad_probs"], score=c["score"], renormalize=c["renorm"],
                                     scale=c["scale"])
    if kind == "w4":
        return ep.ep_expert_matmul_w4(s["x"], s["weights"], s["offsets"], src=s["src"],
                                      rows=s["rows"])
    # rows that no choice names are cleared where there are such rows
    clear = (s["counts"], s["offsets"]) if c["masked"] else None
    if kind == "permute":
        return ep.ep_permute(s["x"], s["slot"], s["weights"], rows=s["rows"], clear=clear)
    if kind == "unpermute":
        return ep.ep_unpermute(s["y"], s["slot"], s["weights"])
    if kind == "permute_bwd":
        gx, gw = ep.ep_permute_backward(s["y"], s["slot"], s["weights"], s["x"])
        return gx if s["weights"] is None else (gx, gw)
    gy, gw = ep.ep_unpermute_backward(s["x"], s["slot"], s["weights"], s["y"], rows=s["rows"],
                                      clear=clear)
    return gy if s["weights"] is None else (gy, gw)


# ------------------------------------------------------------------ the work --

def work(case):
    c = case
    b = _BYTES[c["dtype"]]
    if c["kind"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * b + T * k * 12 + (T * E * 4 if c["probs"] else 0)
                + (E * 4 if c["bias"] else 0), "flops": T * E * (4 + k)}
    if c["kind"] == "router_bwd":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 2 * T * E * b + T * k * 12 + (T * E * 4 if c["probs"] else 0),
                "flops": T * E * 6}
    if c["kind"] == "w4":
        T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
        used = E * (1.0 - (1.0 - k / E) ** T)      # experts that some token chose, on average
        ng = (K + c["group"] - 1) // c["group"]
        per = N * K / 2 + N * ng * (b + (0.5 if c["zeros"] else 0))
        rows_in = T if c["gather"] else T * k
        n_out = N // 2 if c["glu"] else N
        return {"bytes": int(used * per + rows_in * K * b + T * k * n_out * b + 4 * T * k),
                "flops": 2 * T * k * K * N}
    T, H, k = c["T"], c["H"], c["k"]
    pairs = T * k * (1.0 - c["masked"])
    by = T * H * b + pairs * H * b + T * k * 4 * (2 if c["weighted"] else 1)
    flops = pairs * H * 2
    if c["weighted"] and c["kind"] == "permute_bwd":
        by, flops = by + T * H * b + T * k * 4, flops * 2
    if c["kind"] == "unpermute_bwd" and c["weighted"]:
        by, flops = by + pairs * H * b + T * k * 4, flops * 2
    if c["kind"] in ("permute", "unpermute_bwd"):
        by += (T * k - pairs) * H * b              # cleared rows
    return {"bytes": int(by), "flops": int(flops)}


# ------------------------------------------------- the definition in 64 bits --

def _exact_router(s):
    c = s["case"]
    T, E, k = c["T"], c["E"], c["k"]
    L = s["logits"].double()
    live = L > -math.inf
    if c["score"] == "softmax":
        score = torch.exp(L - torch.logsumexp(torch.where(live, L, -1e300), 1, keepdim=True))
        score = torch.where(live, score, 0.0)
    else:
        score = torch.sigmoid(L)
    b = torch.zeros(E, dtype=torch.float64, device=DEV) if s.get("bias") is None else s["bias"].double()
    pick = torch.where(live, score + b if c["bias"] else L, -math.inf)
    value = torch.where(live, score + b, -math.inf)
    if c["groups"] > 1:
        n, per = c["groups"], E // c["groups"]
        src = value if c["bias"] or c["group_top"] > 1 else pick
        rating = torch.full((T, n), -math.inf, dtype=torch.float64, device=DEV)
        for q in range(n):
            part = src[:, q * per:(q + 1) * per].clone()
            total = torch.zeros(T, dtype=torch.float64, device=DEV)
            for r in range(min(c["group_top"], per)):
                v, i = part.max(1)
                total += torch.where(v > -math.inf, v, 0.0)
                if r == 0:
                    seen = v > -math.inf
                part.scatter_(1, i[:, None], -math.inf)
            rating[:, q] = torch.where(seen, total, -math.inf)
        rank = ((rating[:, None, :] > rating[:, :, None])
                | ((rating[:, None, :] == rating[:, :, None])
                   & (torch.arange(n, device=DEV)[None, None, :] < torch.arange(n, device=DEV)[None, :, None]))).sum(2)
        allowed = (rank < c["topk_groups"])[:, torch.arange(E, device=DEV) // per]
        pick = torch.where(allowed, pick, -math.inf)
    idx = torch.full((T, k), -1, dtype=torch.int64, device=DEV)
    left = pick.clone()
    number = torch.arange(E, device=DEV).expand(T, E)
    for j in range(k):
        top = left.max(1, keepdim=True).values
        at = torch.where(left == top, number, E).min(1).values
        has = (top > -math.inf).squeeze(1)
        idx[:, j] = torch.where(has, at, -1)
        left.scatter_(1, at[:, None], -math.inf)
    return score, idx


def _exact_weights(score, idx, c):
    sel = torch.where(idx >= 0, score.gather(1, idx.clamp(min=0)), 0.0)
    if c["renorm"]:
        total = sel.sum(1, keepdim=True)
        sel = torch.where(total > 0, sel / total, 0.0)
    return sel * c["scale"]


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c, kind = case, case["kind"]
    if kind == "router":
        score, idx = _exact_router(s)
        w = _exact_weights(score, idx, c)
        return (idx, w, score) if c["probs"] else (idx, w)
    if kind == "router_bwd":
        # by automatic differentiation of the forward definition
        leaf = s["logits"].double().requires_grad_()
        live = leaf > -math.inf
        if c["score"] == "softmax":
            score = torch.softmax(torch.where(live, leaf, -1e300), 1) * live
        else:
            score = torch.sigmoid(torch.where(live, leaf, 0.0)) * live
        idx = s["topk_idx"]
        sel = torch.where(idx >= 0, score.gather(1, idx.clamp(min=0)), 0.0)
        if c["renorm"]:
            total = sel.sum(1, keepdim=True)
            sel = sel / torch.where(total > 0, total, 1.0)
        loss = (sel * c["scale"] * s["grad_weights"].double()).sum()
        if s["grad_probs"] is not None:
            loss = loss + (score * s["grad_probs"].double()).sum()
        return torch.autograd.grad(loss, leaf)[0]
    if kind == "w4":
        K, N, G = c["K"], c["N"], c["group"]
        ng = (K + G - 1) // G
        out = torch.empty(s["rows"], N, dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            a, b = s["bounds"][e], s["bounds"][e + 1]
            if a == b:
                continue
            rows = s["x"][a:b] if s["src"] is None else s["x"][s["src"][a:b].long()]
            rows = rows.double()
            acc = torch.zeros(b - a, N, dtype=torch.float64, device=DEV)
            for q in range(ng):
                lo, hi = q * G, min(K, (q + 1) * G)
                byte = s["codes"][e][:, lo // 2:hi // 2].to(torch.int32)
                code = torch.empty(N, hi - lo, dtype=torch.float64, device=DEV)
                code[:, 0::2] = (byte % 16).double()
                code[:, 1::2] = (byte // 16).double()
                zero = 8.0 if s["zeros"] is None else s["zeros"][e][:, q].double()
                part = rows[:, lo:hi]
                acc += (part @ code.t() - part.sum(1, keepdim=True) * zero) * s["scales"][e][:, q].double()
            out[a:b] = acc
        if c["glu"]:
            gate, up = out[:, :N // 2], out[:, N // 2:]
            out = gate * torch.sigmoid(gate) * up
        return out
    T, H, k, R = c["T"], c["H"], c["k"], s["rows"]
    slot = s["slot"].reshape(-1).long()
    used = slot >= 0
    pair_of_row = torch.full((R,), -1, dtype=torch.int64, device=DEV)
    pair_of_row[slot[used]] = torch.arange(T * k, device=DEV)[used]
    w = torch.ones(T * k, dtype=torch.float64, device=DEV) if s["weights"] is None \
        else s["weights"].reshape(-1).double()
    row_used = pair_of_row >= 0
    token_of_row = pair_of_row.clamp(min=0) // k
    row_w = torch.where(row_used, w[pair_of_row.clamp(min=0)], 0.0)
    gw = None
    if s["weights"] is not None and kind.endswith("_bwd"):
        dots = (s["x"].double()[token_of_row] * s["y"].double()).sum(1)
        gw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        gw[pair_of_row[row_used]] = dots[row_used]
        gw = gw.reshape(T, k)
        del dots
    if kind in ("permute", "unpermute_bwd"):
        rows = s["x"].double()[token_of_row] * row_w[:, None]
        return rows if gw is None else (rows, gw)
    out = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    out.index_add_(0, token_of_row, s["y"].double() * row_w[:, None])
    return out if gw is None else (out, gw)
