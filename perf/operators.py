"""The serving operators of the MoE library and the cases they are measured on.

Three operators, which a program that serves a mixture-of-experts layer uses together:

 few      the whole layer (router projection, routing, experts, combine) for one to 64 tokens, in bf16
          or fp32, with the weights read once;
 int8     the matrix product of rows quantised to 8-bit integers (one scale a row, found on the fly) with
          8-bit weights (one scale an output channel): one weight, or one for each group of rows;
 layer8   the whole layer with 8-bit weights, for one token up to long prompts.

`own` chooses between the plain form (elementary torch operations in 32 bits) and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
TINY = 2.0 ** -126          # the smallest scale of a quantised row


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one token of a chat turn, router and all: the smallest step of a decoder
        dict(name="few_one_token", op="few", T=1, H=2048, F=768, E=128, El=128, e0=0, k=8, dtype="bf16", router=True,
             zipf=0.0),
        # a small batch of decoding requests
        dict(name="few_batch_8", op="few", T=8, H=2048, F=768, E=128, El=128, e0=0, k=8, dtype="bf16", router=True,
             zipf=0.0),
        # the largest batch, wide experts, a few experts much more popular than the rest, logits already known
        dict(name="few_batch_64_skewed", op="few", T=64, H=4096, F=1536, E=128, El=128, e0=0, k=8, dtype="bf16",
             router=False, zipf=1.1),
        # one rank's share of a small fp32 layer, an odd number of tokens, some of them with no expert here
        dict(name="few_share_fp32", op="few", T=13, H=256, F=128, E=8, El=3, e0=2, k=2, dtype="fp32", router=False,
             zipf=0.0),
        # three rows against one projection: a product that reads the weight and little else
        dict(name="int8_rows_3", op="int8", M=3, N=1536, K=2048, G=1, x="bf16", out="bf16", skew=0.0),
        # a long prompt against one projection
        dict(name="int8_rows_16384", op="int8", M=16384, N=4096, K=2048, G=1, x="bf16", out="bf16", skew=0.0),
        # the down product of 128 experts over the routed pairs of a long prompt, popular experts first
        dict(name="int8_experts", op="int8", M=65536, N=2048, K=768, G=128, x="bf16", out="bf16", skew=1.1),
        # ragged everywhere: odd rows and channels, a contraction that ends inside a tile, empty groups
        dict(name="int8_ragged", op="int8", M=1117, N=777, K=1104, G=9, x="fp32", out="fp32", skew=2.0),
        # one token through the 8-bit layer
        dict(name="layer8_one_token", op="layer8", T=1, H=2048, F=768, E=128, El=128, e0=0, k=8, router=True, zipf=0.0),
        # a batch of decoding requests through the 8-bit layer
        dict(name="layer8_batch_32", op="layer8", T=32, H=2048, F=768, E=128, El=128, e0=0, k=8, router=True, zipf=0.0),
        # one rank's sixteen experts, a prompt of odd length
        dict(name="layer8_share", op="layer8", T=1333, H=2048, F=768, E=128, El=16, e0=16, k=8, router=False, zipf=0.0),
        # a long prompt through the 8-bit layer
        dict(name="layer8_prompt", op="layer8", T=16384, H=2048, F=768, E=128, El=128, e0=0, k=8, router=False,
             zipf=0.0),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _layer_shape(rng, T, weight_bytes, most):
    """Sizes of a layer whose weights stay within `most` bytes and whose work within the listed cases'."""
    while True:
        H, F = 256 * _log(rng, 1, 16), 128 * _log(rng, 1, 12)
        E = _log(rng, 2, 256)
        k = min(E, rng.choice([rng.randint(1, 10), rng.randint(1, 10), _log(rng, 1, 32)]))
        El, e0, zipf = E, 0, rng.choice([0.0, 0.0, 1.1])
        if rng.random() < 0.35:             # one rank's share, of evenly used experts
            El = rng.randint(1, E)
            e0, zipf = rng.randint(0, E - El), 0.0
        if 3 * El * H * F * weight_bytes <= most and T * k * H * F <= 16384 * 8 * 2048 * 768:
            return dict(T=T, H=H, F=F, E=E, El=El, e0=e0, k=k, zipf=zipf)


def draw(rng):
    op = rng.choice(["few", "int8", "layer8"])
    if op == "few":
        c = dict(op=op, **_layer_shape(rng, _log(rng, 1, 64), 2, 4.5e9))
        c["dtype"] = "fp32" if 3 * c["El"] * c["H"] * c["F"] < 4e8 and rng.random() < 0.25 else "bf16"
        c["router"] = rng.random() < 0.5
        return c
    if op == "int8":
        while True:
            c = dict(op=op, M=_log(rng, 1, 65536), N=_log(rng, 1, 4096), K=16 * _log(rng, 1, 256),
                     G=rng.choice([1, 1, _log(rng, 2, 160)]))
            if c["M"] * c["N"] * c["K"] <= 16384 * 4096 * 2048 and c["G"] * c["N"] * c["K"] <= 4e8:
                break
        c["x"], c["out"] = rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["bf16", "bf16", "fp32"])
        c["skew"] = rng.choice([0.0, 1.1, 2.0]) if c["G"] > 1 else 0.0
        return c
    c = dict(op=op, **_layer_shape(rng, _log(rng, 1, 16384), 1, 1.3e9))
    c["router"] = rng.random() < 0.5
    return c


def _dtype(name):
    return {"bf16": torch.bfloat16, "fp32": torch.float32}[name]


# ------------------------------------------------------------------------------------------------ inputs

def _quantise_weight(w):
    """8-bit weight with one scale an output channel: w [.., N, K] -> (int8 [.., N, K], float32 [.., N])."""
    scale = (w.float().abs().amax(-1) / 127.0).clamp_min(TINY)
    return (w.float() / scale[..., None]).round().clamp(-127, 127).to(torch.int8), scale


def _normal(g, shape, std, dtype):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _weights(g, El, rows, cols, dtype, quantised):
    """Expert weights [El, rows, cols], filled a few experts at a time; 8-bit as (int8, scales)."""
    w = torch.empty(El, rows, cols, dtype=torch.int8 if quantised else dtype, device=DEV)
    s = torch.empty(El, rows, dtype=torch.float32, device=DEV) if quantised else None
    step = max(1, (1 << 26) // (rows * cols))
    for e in range(0, El, step):
        part = _normal(g, (min(step, El - e), rows, cols), 1.0 / math.sqrt(cols), torch.bfloat16 if quantised else dtype)
        if quantised:
            w[e:e + step], s[e:e + step] = _quantise_weight(part)
        else:
            w[e:e + step] = part
    return (w, s) if quantised else w


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1))
    st = dict(case)
    if case["op"] == "int8":
        M, N, K, G = case["M"], case["N"], case["K"], case["G"]
        # activations have rows of very different size
        size = torch.exp(torch.randn((M, 1), generator=g, device=DEV))
        st["x"] = (torch.randn((M, K), generator=g, device=DEV) * size).to(_dtype(case["x"]))
        w, s = _weights(g, G, N, K, torch.bfloat16, True)
        st["w"], st["ws"] = (w, s) if G > 1 else (w[0], s[0])
        if G > 1:
            p = torch.arange(1, G + 1, device=DEV, dtype=torch.float32) ** -case["skew"]
            group = torch.multinomial(p / p.sum(), M, replacement=True, generator=g)
            counts = torch.bincount(group, minlength=G)
            st["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        else:
            st["offsets"] = None
        if own:
            import mixture_experts_layer_32_amd.layer as L
            st["call"] = L
        return st
    T, H, F, E, El = (case[n] for n in ("T", "H", "F", "E", "El"))
    dt = _dtype(case.get("dtype", "bf16"))
    q = case["op"] == "layer8"
    st["x"] = _normal(g, (T, H), 1.0, dt)
    wr = _normal(g, (E, H), 0.02, dt)
    if case["zipf"] > 0 and not case["router"]:
        prior = -case["zipf"] * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float64))
    else:
        prior = 0.0
    st["wr"] = wr if case["router"] else None
    st["logits"] = None if case["router"] else (st["x"].double() @ wr.double().T + prior).float()
    st["wg"] = _weights(g, El, F, H, dt, q)
    st["wu"] = _weights(g, El, F, H, dt, q)
    st["wd"] = _weights(g, El, H, F, dt, q)
    if own:
        import mixture_experts_layer_32_amd.layer as L
        st["call"] = (L.Int8Layer(T, H, F, E, case["k"], E_local=El, expert_offset=case["e0"]) if q else
                      L.FewTokenLayer(T, H, F, E, case["k"], case["dtype"], E_local=El, expert_offset=case["e0"]))
    return st


# ------------------------------------------------------------------------------------------------ plain form

def _quantise_rows(x):
    """Rows of x as whole numbers of -127..127 (in fp32) and one scale a row. The quotient is taken in 64
    bits: bf16 rows hold values halfway between two whole numbers (half of the row's largest, for one)."""
    most = x.float().abs().amax(-1).clamp_min(127.0 * TINY)
    return (127.0 * x.double() / most.double()[:, None]).round().float(), most / 127.0


def _by_expert(e, El, P):
    """Tiles of rows that share an expert: the tile rows' source order and slots, and each tile's expert.
    e [P]: the row's expert, El for none. The number of tiles is bounded by the sizes alone."""
    r = 16 if P < 64 * El else 128
    nt = min(P, P // r + El + 1)
    order = torch.sort(e, stable=True).indices
    es = e[order]
    counts = torch.zeros(El + 1, dtype=torch.int64, device=e.device).scatter_add_(0, e, torch.ones_like(e))
    tiles = (counts + r - 1) // r
    first_row, first_tile = counts.cumsum(0) - counts, tiles.cumsum(0) - tiles
    slot = first_tile[es] * r + torch.arange(P, device=e.device) - first_row[es]
    expert = torch.searchsorted(tiles.cumsum(0), torch.arange(nt, device=e.device), right=True).clamp(max=El - 1)
    return r, nt, order, slot, expert


def _product(plan, a, w):
    """Rows of a, in the plan's order, times their expert's w [El, N, K]: [P, N] in fp32."""
    r, nt, _, slot, expert = plan
    buf = torch.zeros(nt * r, a.shape[1], dtype=torch.float32, device=a.device)
    buf[slot] = a.float()
    return torch.bmm(buf.view(nt, r, -1), w[expert].float().transpose(1, 2)).view(nt * r, -1)[slot]


def _route(logits, k):
    v, i = torch.sort(logits.float(), dim=-1, descending=True, stable=True)
    v, i = v[:, :k], i[:, :k]
    z = torch.exp(v - v[:, :1])
    return i, z / z.sum(-1, keepdim=True)


def _layer(st, quantised):
    """The layer's y, from 8-bit weights with both products' rows quantised where `quantised`."""
    x, k, El, e0 = st["x"], st["k"], st["El"], st["e0"]
    T, H = x.shape
    logits = st["logits"] if st["wr"] is None else x.float() @ st["wr"].float().T
    idx, weight = _route(logits, k)
    el = idx.reshape(-1) - e0
    here = (el >= 0) & (el < El)
    plan = _by_expert(torch.where(here, el, El), El, T * k)
    order, expert = plan[2], torch.where(here, el, 0)[plan[2]]
    tok, wt = order // k, weight.reshape(-1)[order]
    if quantised:
        (wg, sg), (wu, su), (wd, sd) = st["wg"], st["wu"], st["wd"]
        xq, xs = _quantise_rows(x)
        a = _product(plan, xq[tok], wg) * (xs[tok][:, None] * sg[expert])
        b = _product(plan, xq[tok], wu) * (xs[tok][:, None] * su[expert])
        hq, hs = _quantise_rows(wt[:, None] * (a / (1.0 + torch.exp(-a)) * b))
        o = _product(plan, hq, wd) * (hs[:, None] * sd[expert])
    else:
        a, b = _product(plan, x[tok], st["wg"]), _product(plan, x[tok], st["wu"])
        o = _product(plan, wt[:, None] * (a / (1.0 + torch.exp(-a)) * b), st["wd"])
    pairs = torch.empty_like(o)
    pairs[order] = torch.where(here[order][:, None], o, 0.0)
    y = pairs.view(T, k, H).sum(1).to(x.dtype)
    return y if st["wr"] is None else (y, logits)


def _int8(st):
    x, w, ws, offsets = st["x"], st["w"], st["ws"], st["offsets"]
    q, s = _quantise_rows(x)
    out = _dtype(st["out"])
    if offsets is None:
        return ((q @ w.float().T) * (s[:, None] * ws)).to(out)
    G = w.shape[0]
    e = torch.searchsorted(offsets[1:].long(), torch.arange(x.shape[0], device=x.device), right=True)
    plan = _by_expert(e, G, x.shape[0])
    return (_product(plan, q, w) * (s[:, None] * ws[e])).to(out)


# ------------------------------------------------------------------------------------------------ one pass

def run(st):
    if not own:
        return _int8(st) if st["op"] == "int8" else _layer(st, st["op"] == "layer8")
    call = st["call"]
    if st["op"] == "int8":
        xq, xs = call.int8_quantize(st["x"])
        return call.int8_matmul(xq, xs, st["w"], st["ws"], offsets=st["offsets"], dtype=_dtype(st["out"]))
    if st["wr"] is not None:
        return call.forward_router(st["x"], st["wr"], st["wg"], st["wu"], st["wd"])
    return call.forward(st["x"], st["logits"], st["wg"], st["wu"], st["wd"])


# ------------------------------------------------------------------------------------------------ work

def _active(c):
    """(experts with at least one pair, pairs) here, of a routing of this shape drawn at random."""
    g = torch.Generator().manual_seed(7)
    logits = torch.randn((c["T"], c["E"]), generator=g) * 0.02 * math.sqrt(c["H"])
    if c["zipf"] > 0 and not c["router"]:
        logits -= c["zipf"] * torch.log(torch.arange(1, c["E"] + 1, dtype=torch.float32))
    idx = logits.topk(c["k"], -1).indices.reshape(-1) - c["e0"]
    idx = idx[(idx >= 0) & (idx < c["El"])]
    return int(torch.unique(idx).numel()), int(idx.numel())


def work(case):
    c = case
    if c["op"] == "int8":
        xb, ob = (2 if c["x"] == "bf16" else 4), (2 if c["out"] == "bf16" else 4)
        groups = min(c["G"], c["M"])
        return {"bytes": c["M"] * c["K"] * xb + groups * c["N"] * (c["K"] + 4) + c["M"] * c["N"] * ob,
                "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    experts, pairs = _active(c)
    q = c["op"] == "layer8"
    eb = 4 if c.get("dtype") == "fp32" else 2
    wb = 1 if q else eb
    T, H, F, E = c["T"], c["H"], c["F"], c["E"]
    return {"bytes": 2 * T * H * eb + 4 * T * E + (E * H * eb if c["router"] else 0) +
                     experts * (3 * H * F * wb + (4 * (2 * F + H) if q else 0)),
            "flops": 6.0 * pairs * H * F + (2.0 * T * E * H if c["router"] else 0)}


# ------------------------------------------------------------------------------------------------ 64 bits

def _quantise_rows64(x):
    most = torch.clamp(x.abs().max(dim=1).values, min=127 * TINY)
    return torch.round(x * 127 / most[:, None]), most / 127


def exact(case, seed):
    st = prepare(case, seed)
    x = st["x"].double()
    if case["op"] == "int8":
        q, s = _quantise_rows64(x)
        if st["offsets"] is None:
            return (q @ st["w"].double().T) * s[:, None] * st["ws"].double()
        bounds, y = st["offsets"].tolist(), torch.empty(case["M"], case["N"], dtype=torch.float64, device=DEV)
        for e in range(case["G"]):
            a, b = bounds[e], bounds[e + 1]
            y[a:b] = (q[a:b] @ st["w"][e].double().T) * s[a:b, None] * st["ws"][e].double()
        return y
    quantised = case["op"] == "layer8"
    logits = st["logits"].double() if st["wr"] is None else x @ st["wr"].double().T
    chosen = torch.argsort(-logits, dim=1, stable=True)[:, :case["k"]]
    weight = torch.softmax(torch.gather(logits, 1, chosen), 1)
    y = torch.zeros_like(x)
    xq, xs = _quantise_rows64(x) if quantised else (x, None)
    for e in range(case["El"]):
        t, j = torch.nonzero(chosen == case["e0"] + e, as_tuple=True)
        if t.numel() == 0:
            continue
        if quantised:
            (wg, sg), (wu, su), (wd, sd) = ((m[0][e].double(), m[1][e].double()) for m in (st["wg"], st["wu"], st["wd"]))
            a, b = (xq[t] @ wg.T) * xs[t, None] * sg, (xq[t] @ wu.T) * xs[t, None] * su
            hq, hs = _quantise_rows64(weight[t, j, None] * a * torch.sigmoid(a) * b)
            o = (hq @ wd.T) * hs[:, None] * sd
        else:
            a, b = x[t] @ st["wg"][e].double().T, x[t] @ st["wu"][e].double().T
            o = (weight[t, j, None] * a * torch.sigmoid(a) * b) @ st["wd"][e].double().T
        y.index_add_(0, t, o)
    return y if st["wr"] is None else (y, logits)
