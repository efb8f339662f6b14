"""More operators of the MoE library and the cases they are measured on.

What a program uses that takes the layer apart (experts of its own, weights in 4 bits) or trains it:

 dispatch   the routed (token, slot) pairs sorted by expert, and the tokens' rows brought into that order
 combine    the pairs' rows brought back to their tokens, multiplied with the routing weights and added up
 gradients  of both: of the pairs' rows, the routing weights, the router's logits and the tokens
 int4       the product of bf16 rows with 4-bit weights that have a scale for each group of inputs: one
            weight, or one for each group of rows
 clip       the norm over all gradients together, and the gradients scaled so that it stays within a bound

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a small batch of decoding requests, sorted by expert
        dict(name="dispatch_batch_8", op="dispatch", T=8, H=2048, k=8, E=128, El=128, e0=0, dtype="bf16", zipf=0.0,
             drop=0.0),
        # a long prompt or a training sequence
        dict(name="dispatch_prompt", op="dispatch", T=16384, H=2048, k=8, E=128, El=128, e0=0, dtype="bf16", zipf=0.0,
             drop=0.0),
        # one token's pairs back together: the smallest step of a decoder
        dict(name="combine_one_token", op="combine", T=1, H=2048, k=8, E=128, El=128, e0=0, rows="fp32", dtype="bf16",
             zipf=0.0, drop=0.0, weighted=True),
        # a training sequence, popular experts first
        dict(name="combine_prompt", op="combine", T=16384, H=2048, k=8, E=128, El=128, e0=0, rows="bf16", dtype="bf16",
             zipf=1.1, drop=0.0, weighted=True),
        # the backward pass of a training sequence
        dict(name="gradients_train", op="gradients", T=16384, H=2048, k=8, E=128, El=128, e0=0, rows="bf16",
             dtype="bf16", zipf=0.0, drop=0.0, logits=True),
        # one rank's sixteen experts, odd numbers of tokens and features, tokens without any pair here
        dict(name="gradients_share_fp32", op="gradients", T=1333, H=1001, k=6, E=128, El=16, e0=16, rows="fp32",
             dtype="fp32", zipf=0.0, drop=0.1, logits=True),
        # one row against one projection: the weight read once and little else
        dict(name="int4_one_row", op="int4", M=1, N=1536, K=4096, G=1, group=128, out="bf16", skew=0.0),
        # eight decoding requests at eight experts each: a row or two for half of the experts
        dict(name="int4_experts_batch", op="int4", M=64, N=1536, K=4096, G=128, group=128, out="bf16", skew=0.0),
        # ragged everywhere: odd rows and channels, inputs that end inside a tile, popular groups, empty ones
        dict(name="int4_ragged", op="int4", M=1117, N=777, K=1120, G=9, group=32, out="fp32", skew=2.0),
        # a long prompt against one projection
        dict(name="int4_prompt", op="int4", M=16384, N=4096, K=2048, G=1, group=64, out="bf16", skew=0.0),
        # a layer's gradients: three of its 128 experts' and the router's, into buffers for the optimizer, clipped
        dict(name="clip_layer", op="clip", sizes="layer", count=4, total=3 * 128 * 768 * 2048 + 128 * 2048,
             dtype="bf16", place=False, over=True),
        # many small gradients of both types, in place, within the bound
        dict(name="clip_small", op="clip", sizes="spread", count=150, total=400000, dtype="both", place=True,
             over=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _pairs_shape(rng):
    while True:
        T, H, E = _log(rng, 1, 16384), _log(rng, 1, 8192), _log(rng, 1, 512)
        if rng.random() < 0.6:
            H = max(8, H // 8 * 8)
        k = min(E, rng.choice([rng.randint(1, 10), _log(rng, 1, 32)]))
        El, e0, zipf = E, 0, rng.choice([0.0, 0.0, 1.1])
        if rng.random() < 0.35:             # one rank's share
            El = rng.randint(1, E)
            e0, zipf = rng.randint(0, E - El), 0.0
        if T * k * H <= 16384 * 8 * 2048 and T * E <= 16384 * 128:
            return dict(T=T, H=H, k=k, E=E, El=El, e0=e0, zipf=zipf, drop=rng.choice([0.0, 0.0, 0.2]))


def draw(rng):
    op = rng.choice(["dispatch", "combine", "gradients", "int4", "int4", "clip"])
    if op == "dispatch":
        return dict(op=op, **_pairs_shape(rng), dtype=rng.choice(["bf16", "bf16", "fp32", "int8"]))
    if op in ("combine", "gradients"):
        c = dict(op=op, **_pairs_shape(rng))
        c["rows"], c["dtype"] = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16")])
        if "fp32" in c["rows"]:
            c["T"] = max(1, c["T"] // 2)
        c["weighted" if op == "combine" else "logits"] = rng.random() < 0.7
        return c
    if op == "int4":
        while True:
            group = rng.choice([32, 64, 128])
            c = dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 1, 4096), K=group * _log(rng, 1, 8192 // group),
                     G=rng.choice([1, 1, _log(rng, 2, 160)]), group=group)
            tiles = c["M"] // 16 + c["G"] + 1 if c["M"] < 64 * c["G"] else c["M"] // 128 + c["G"] + 1
            if c["M"] * c["N"] * c["K"] <= 16384 * 4096 * 2048 and c["G"] * c["N"] * c["K"] <= 8e8 and (
                    c["G"] == 1 or tiles * c["N"] * c["K"] <= 1.5e9):
                break
        c["out"] = rng.choice(["bf16", "bf16", "fp32"])
        c["skew"] = rng.choice([0.0, 1.1, 2.0]) if c["G"] > 1 else 0.0
        return c
    count = _log(rng, 1, 300)
    place = rng.random() < 0.4
    return dict(op=op, sizes="spread", count=count, total=max(count, _log(rng, 100, 300000000)),
                dtype=rng.choice(["bf16", "fp32", "both"]), place=place, over=not place and rng.random() < 0.7)


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32, "int8": torch.int8}[name]


# ------------------------------------------------------------------------------------------------ inputs

def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _routing(g, c):
    """The router's choice: idx [T, k] int32 (-1 for a pair that was dropped) and weights [T, k] fp32."""
    logits = torch.randn((c["T"], c["E"]), generator=g, device=DEV)
    if c["zipf"] > 0:
        logits -= c["zipf"] * torch.log(torch.arange(1, c["E"] + 1, device=DEV, dtype=torch.float32))
    v, i = torch.sort(logits, dim=-1, descending=True, stable=True)
    weight = torch.softmax(v[:, :c["k"]], dim=-1).contiguous()
    idx = i[:, :c["k"]].to(torch.int32)
    gone = torch.rand(idx.shape, generator=g, device=DEV) < c["drop"]
    return torch.where(gone, -1, idx).contiguous(), weight


def _sorted_pairs(idx, c):
    """(offsets [El + 1], perm [T k], pair_pos [T, k]), int32: pairs ordered by expert, then by number."""
    e = idx.reshape(-1).long() - c["e0"]
    e = torch.where((e >= 0) & (e < c["El"]), e, c["El"])
    order = torch.sort(e, stable=True).indices
    counts = torch.zeros(c["El"] + 1, dtype=torch.int64, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    offsets = counts.cumsum(0) - counts
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=e.device)
    here = e < c["El"]
    return (offsets.to(torch.int32), torch.where(here[order], order, -1).to(torch.int32),
            torch.where(here, pos, -1).to(torch.int32).view(idx.shape))


def _sizes(c):
    if c["sizes"] == "layer":
        return [128 * 768 * 2048] * 3 + [128 * 2048]
    # a few large tensors and many small ones, odd sizes among them, some empty
    share = [1.0 / (1 + i) for i in range(c["count"])]
    return [0 if i % 29 == 28 else max(1, int(c["total"] * s / sum(share))) for i, s in enumerate(share)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1))
    st = dict(case)
    call = None
    if own:
        import mixture_experts_layer_32_amd.layer as call
        st["call"] = call
    if case["op"] == "clip":
        sizes = _sizes(case)
        kinds = ["bf16", "fp32"][:len(sizes)] if case["dtype"] == "both" else [case["dtype"]]
        flat, grads, out = [], [None] * len(sizes), [None] * len(sizes)
        # the gradients of a type lie one behind the other in one buffer, as a framework's buckets hold them
        for b, kind in enumerate(kinds):
            mine = range(b, len(sizes), len(kinds))
            buf = torch.empty(sum(sizes[i] for i in mine), dtype=_dtype(kind), device=DEV)
            to, at = buf if case["place"] else torch.empty_like(buf), 0
            for i in mine:
                grads[i], out[i] = buf[at:at + sizes[i]], to[at:at + sizes[i]]
                at += sizes[i]
                for a in range(0, sizes[i], 1 << 26):     # gradients of very different size
                    part = grads[i][a:a + (1 << 26)]
                    part.copy_(_normal(g, part.shape, 10.0 ** (-2 - i % 4), buf.dtype))
            flat.append(to)
        st["grads"], st["out"], st["flat"] = grads, out, flat
        expected = math.sqrt(sum(n * 10.0 ** (2 * (-2 - i % 4)) for i, n in enumerate(sizes)))
        st["max_norm"] = expected * (0.3 if case["over"] else 3.0)
        if own:
            st["plan"] = call.GradNorm(grads, None if case["place"] else out)
        return st
    if case["op"] == "int4":
        M, N, K, G, group = (case[n] for n in ("M", "N", "K", "G", "group"))
        # activations have rows of very different size
        size = torch.exp(torch.randn((M, 1), generator=g, device=DEV))
        st["x"] = (torch.randn((M, K), generator=g, device=DEV) * size).to(torch.bfloat16)
        q = torch.empty((G, N, K), dtype=torch.int8, device=DEV)
        s = torch.empty((G, N, K // group), dtype=torch.bfloat16, device=DEV)
        step = max(1, (1 << 26) // (N * K))
        for e in range(0, G, step):
            w = _normal(g, (min(step, G - e), N, K // group, group), 1.0 / math.sqrt(K), torch.float32)
            s[e:e + step] = (w.abs().amax(-1) / 7.0).to(torch.bfloat16)
            q[e:e + step] = (w / s[e:e + step, ..., None].float()).round().clamp(-8, 7).to(torch.int8).view(-1, N, K)
        st["q"], st["s"] = (q, s) if G > 1 else (q[0], s[0])
        if G > 1:
            p = torch.arange(1, G + 1, device=DEV, dtype=torch.float32) ** -case["skew"]
            chosen = torch.multinomial(p / p.sum(), M, replacement=True, generator=g)
            counts = torch.bincount(chosen, minlength=G)
            st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        else:
            st["offsets"] = None
        if own:
            st["w"] = call.int4_pack(st["q"], st["s"])
        return st
    T, H, k = case["T"], case["H"], case["k"]
    st["idx"], st["weight"] = _routing(g, case)
    dt = _dtype(case["dtype"])
    if case["op"] == "dispatch":
        x = torch.randn((T, H), generator=g, device=DEV)
        st["x"] = (x * 30).round().clamp(-127, 127).to(dt) if dt == torch.int8 else x.to(dt)
        st["rows"] = torch.zeros((T * k, H), dtype=dt, device=DEV)
        return st
    _, _, st["pair_pos"] = _sorted_pairs(st["idx"], case)
    rt = _dtype(case["rows"])
    st["rows"] = _normal(g, (T * k, H), 1.0, rt)
    if case["op"] == "combine":
        st["weight"] = st["weight"] if case["weighted"] else None
        return st
    st["dy"] = _normal(g, (T, H), 0.01, dt)
    st["dsorted"] = _normal(g, (T * k, H), 0.01, rt)
    st["drows"] = torch.zeros((T * k, H), dtype=rt, device=DEV)
    return st


# ------------------------------------------------------------------------------------------------ plain form

def _by_group(offsets, M):
    """Tiles of rows that share a group: each row's slot, and each tile's group. The number of tiles is
    bounded by the sizes alone."""
    G = offsets.numel() - 1
    r = 16 if M < 64 * G else 128
    nt = min(M, M // r + G + 1)
    off = offsets.long()
    row = torch.arange(M, device=off.device)
    e = torch.searchsorted(off[1:], row, right=True)
    tiles = (off[1:] - off[:-1] + r - 1) // r
    slot = (tiles.cumsum(0) - tiles)[e] * r + row - off[e]
    return r, nt, slot, torch.searchsorted(tiles.cumsum(0), torch.arange(nt, device=off.device), right=True).clamp(max=G - 1)


def _int4(st):
    x, q, s, offsets, group = st["x"].float(), st["q"], st["s"], st["offsets"], st["group"]
    out = _dtype(st["out"])

    def weight(q, s):
        return (q.float().unflatten(-1, (-1, group)) * s.float()[..., None]).flatten(-2)
    if offsets is None:
        return (x @ weight(q, s).T).to(out)
    r, nt, slot, tile = _by_group(offsets, x.shape[0])
    buf = torch.zeros(nt * r, x.shape[1], device=x.device)
    buf[slot] = x
    y = torch.bmm(buf.view(nt, r, -1), weight(q[tile], s[tile]).transpose(1, 2))
    return y.view(nt * r, -1)[slot].to(out)


def _dispatch(st):
    offsets, perm, pair_pos = _sorted_pairs(st["idx"], st)
    rows = torch.where(perm[:, None] >= 0, st["x"][perm.clamp(min=0).long() // st["k"]], 0)
    return offsets, perm, pair_pos, rows


def _combine(rows, pair_pos, weight, dtype):
    here = pair_pos >= 0
    v = rows[pair_pos.clamp(min=0).long()].float()
    if weight is not None:
        v = v * weight[..., None]
    return torch.where(here[..., None], v, 0.0).sum(1).to(dtype)


def _gradients(st):
    dy, rows, pair_pos, weight, idx = st["dy"].float(), st["rows"], st["pair_pos"], st["weight"], st["idx"].long()
    here = pair_pos >= 0
    drows = torch.zeros((rows.shape[0] + 1, rows.shape[1]), dtype=rows.dtype, device=rows.device)
    to = torch.where(here, pair_pos.long(), rows.shape[0])
    dweight = torch.empty_like(weight)
    for j in range(st["k"]):
        drows[to[:, j]] = (weight[:, j, None] * dy).to(rows.dtype)
        dot = (dy * rows[pair_pos[:, j].clamp(min=0).long()].float()).sum(-1)
        dweight[:, j] = torch.where(here[:, j], dot, 0.0)
    dx = _combine(st["dsorted"], pair_pos, None, st["dy"].dtype)
    if not st["logits"]:
        return drows[:-1], dweight, dx
    dl = weight * (dweight - (weight * dweight).sum(-1, keepdim=True))
    dlogits = torch.zeros((dy.shape[0], st["E"] + 1), device=dy.device)
    dlogits.scatter_(1, torch.where(idx >= 0, idx, st["E"]), dl)
    return drows[:-1], dweight, dlogits[:, :-1].contiguous(), dx


def _clip(st):
    total = sum((t.double() ** 2).sum() for t in st["grads"])
    norm = total.sqrt().float()
    c = (st["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    for t, o in zip(st["grads"], st["out"]):
        o.copy_(t.float() * c)
    return norm, st["flat"]


# ------------------------------------------------------------------------------------------------ one pass

def run(st):
    op = st["op"]
    if not own:
        if op == "dispatch":
            return _dispatch(st)
        if op == "combine":
            return _combine(st["rows"], st["pair_pos"], st["weight"], _dtype(st["dtype"]))
        return {"gradients": _gradients, "int4": _int4, "clip": _clip}[op](st)
    call = st["call"]
    if op == "dispatch":
        offsets, perm, pair_pos = call.sort_pairs(st["idx"], st["El"], st["e0"])
        return offsets, perm, pair_pos, call.dispatch(st["x"], pair_pos, rows=st["rows"])
    if op == "combine":
        return call.combine(st["rows"], st["pair_pos"], st["weight"], dtype=_dtype(st["dtype"]))
    if op == "gradients":
        out = call.combine_backward(st["dy"], st["rows"], st["weight"], st["pair_pos"],
                                    idx=st["idx"] if st["logits"] else None,
                                    E_total=st["E"] if st["logits"] else None, drows=st["drows"])
        return (*out, call.combine(st["dsorted"], st["pair_pos"], dtype=_dtype(st["dtype"])))
    if op == "int4":
        return call.int4_matmul(st["x"], *st["w"], offsets=st["offsets"], N=st["N"], dtype=_dtype(st["out"]))
    return st["plan"].clip(st["max_norm"]), st["flat"]


# ------------------------------------------------------------------------------------------------ work

def work(case):
    c, size = case, {"bf16": 2, "fp32": 4, "int8": 1}
    if c["op"] == "clip":
        sizes = _sizes(c)
        eb = [size[c["dtype"]] if c["dtype"] != "both" else (2, 4)[i % 2] for i in range(len(sizes))]
        n = sum(a * b for a, b in zip(sizes, eb))
        # the norm needs every gradient before the first can be scaled
        passes = (2 if c["over"] else 1) + (0 if c["place"] and not c["over"] else 1)
        return {"bytes": passes * n, "flops": 3.0 * sum(sizes)}
    if c["op"] == "int4":
        groups = min(c["G"], c["M"])
        return {"bytes": 2 * c["M"] * c["K"] + groups * c["N"] * (c["K"] / 2 + 2 * c["K"] / c["group"]) +
                         c["M"] * c["N"] * size[c["out"]], "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    T, H, k = c["T"], c["H"], c["k"]
    pairs = max(1.0, T * k * c["El"] / c["E"] * (1 - c["drop"]))
    eb = size[c["dtype"]]
    if c["op"] == "dispatch":
        return {"bytes": 12 * T * k + T * H * eb + pairs * H * eb, "flops": T * k}
    rb = size[c["rows"]]
    if c["op"] == "combine":
        return {"bytes": 8 * T * k + T * H * eb + pairs * H * rb, "flops": 2.0 * pairs * H}
    return {"bytes": 16 * T * k + 2 * T * H * eb + 3 * pairs * H * rb + (4 * T * c["E"] if c["logits"] else 0),
            "flops": 4.0 * pairs * H}


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "clip":
        norm = torch.sqrt(sum(torch.linalg.vector_norm(t, dtype=torch.float64) ** 2 for t in st["grads"]))
        f = torch.clamp(st["max_norm"] / (norm + 1e-6), max=1.0)
        kinds = [[t for t in st["grads"] if t.dtype == to.dtype] for to in st["flat"]]
        return norm, [torch.cat([t.double() * f for t in ts]) for ts in kinds]
    if case["op"] == "int4":
        G, group = case["G"], case["group"]
        q, s = (st["q"], st["s"]) if G > 1 else (st["q"][None], st["s"][None])
        bounds = st["offsets"].tolist() if G > 1 else [0, case["M"]]
        y = torch.empty(case["M"], case["N"], dtype=torch.float64, device=DEV)
        for e in range(G):
            a, b = bounds[e], bounds[e + 1]
            if a < b:
                y[a:b] = st["x"][a:b].double() @ (q[e].double() * torch.repeat_interleave(s[e].double(), group, dim=1)).T
        return y
    T, H, k = case["T"], case["H"], case["k"]
    e = st["idx"].flatten().long() - case["e0"]
    local = (e >= 0) & (e < case["El"])
    pairs = torch.nonzero(local).flatten()
    pairs = pairs[torch.argsort(e[pairs] * (T * k) + pairs)]
    token = pairs // k
    P = pairs.numel()
    if case["op"] == "dispatch":
        perm = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
        perm[:P] = pairs.to(torch.int32)
        pair_pos = torch.full((T * k,), -1, dtype=torch.int32, device=DEV)
        pair_pos[pairs] = torch.arange(P, device=DEV, dtype=torch.int32)
        offsets = torch.searchsorted(e[pairs], torch.arange(case["El"] + 1, device=DEV)).to(torch.int32)
        rows = torch.zeros((T * k, H), dtype=torch.float64, device=DEV)
        rows[:P] = st["x"].double()[token]
        return offsets, perm, pair_pos.view(T, k), rows
    if case["op"] == "combine":
        w = torch.ones(P, dtype=torch.float64, device=DEV) if st["weight"] is None else st["weight"].double().flatten()[pairs]
        return torch.zeros((T, H), dtype=torch.float64, device=DEV).index_add_(0, token, st["rows"][:P].double() * w[:, None])
    w, dy = st["weight"].double(), st["dy"].double()
    drows = torch.zeros((T * k, H), dtype=torch.float64, device=DEV)
    drows[:P] = dy[token] * w.flatten()[pairs][:, None]
    dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
    dw[pairs] = torch.einsum("ph,ph->p", dy[token], st["rows"][:P].double())
    dw = dw.view(T, k)
    dx = torch.zeros((T, H), dtype=torch.float64, device=DEV).index_add_(0, token, st["dsorted"][:P].double())
    if not case["logits"]:
        return drows, dw, dx
    jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]      # of the softmax over the chosen experts
    dl = (jac * dw[:, None, :]).sum(-1)
    full = torch.zeros((T, case["E"]), dtype=torch.float64, device=DEV)
    t, j = torch.nonzero(st["idx"] >= 0, as_tuple=True)
    full[t, st["idx"][t, j].long()] = dl[t, j]
    return drows, dw, full, dx
