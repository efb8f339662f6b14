"""GPU: 8-bit rows (moe_int8_quantize), products (moe_int8_matmul) and the 8-bit layer (moe_fwd_int8).

The quantiser and the product are compared bit for bit with their definitions in 64 bits (numpy). The layer
is compared with the same steps in float64. Its bars, relative Frobenius: y is rounded to bf16 once, by at
most 2^-8 of each value (up to 64 tokens), or each pair's output and y are (more tokens: 2 * 2^-8); h's
fp32 error (about 2^-22 of a value of up to 127 steps) moves about one in 10^4 of its bytes by one step of
1/127 of the row's largest, less than 1e-3 in all. These bars leave room for a rounding of each pair's output that the
layer does not make; test_layer_is_rounded_once holds every token to one rounding.
"""
import threading

import numpy as np
import pytest
import torch

import oracle
from mixture_experts_layer_32_amd import inputs
from mixture_experts_layer_32_amd.layer import FewTokenLayer, Int8Layer, int8_matmul, int8_quantize
from gpu_util import to_dev
from rounding import BAR, excess

pytestmark = pytest.mark.gpu

FLOOR = np.float32(127.0) * np.float32(2.0) ** np.float32(-126)


def quant_ref(x):
    """(q, fp32 scales) of the rows of a float32 array, by the definition in 64 bits."""
    x = np.asarray(x, np.float32)
    bad = ~np.isfinite(x).all(-1)
    v = np.where(bad[..., None], 0, x).astype(np.float64)
    D = np.maximum(np.abs(v).max(-1), float(FLOOR))
    q = np.rint(127.0 * v / D[..., None]).astype(np.int8)
    s = D.astype(np.float32) / np.float32(127)
    s[bad] = np.nan
    q[bad] = 0
    return q, s


def check_quant(x, dt):
    t = torch.from_numpy(x).to("cuda").to(dt)
    q, s = int8_quantize(t)
    torch.cuda.synchronize()
    rq, rs = quant_ref(t.float().cpu().numpy())
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True)
    assert np.array_equal(q.cpu().numpy(), rq)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 528), (1000, 512), (6, 256), (5, 768), (13, 1008), (77, 1040), (3, 1536), (5, 2048), (9, 4096), (2, 4112),
                                       (1, 131072), (4099, 48)])
def test_quantise_bit_exact(rows, cols, dt):
    print("case int8 quant", rows, cols, dt, flush=True)
    rng = np.random.default_rng(rows * 7 + cols)
    x = rng.standard_normal((rows, cols)).astype(np.float32) * np.exp(rng.standard_normal((rows, 1)) * 4).astype(np.float32)
    check_quant(x, dt)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_quantise_edges(dt):
    """Ties, zeros, the type's ends, subnormals, infinities and NaN."""
    print("case int8 quant edges", dt, flush=True)
    rng = np.random.default_rng(5)
    rows = [np.zeros(256), np.full(256, -3.0)]
    for top in (1.0, 127.0, 254.0, 1.9921875, 3.0e38, 2.0 ** 100, 2.0 ** 120, 1e-37, 2.0 ** -126, 2.0 ** -130, 3e-39):
        n = np.arange(-127, 128, dtype=np.float64)
        r = np.zeros(256)
        r[:255] = (n + 0.5 * (np.arange(255) % 2)) / 127.0 * top       # whole and half steps
        r[np.abs(r) > top] = top / 2                                   # 63.5: a tie in every type
        r[255] = top
        rows.append(r)
    rows.append(rng.standard_normal(256) * 2.0 ** -128)
    for v in (np.nan, np.inf, -np.inf):
        r = rng.standard_normal(256)
        r[rng.integers(256)] = v
        rows.append(r)
    r = np.full(256, 1e30)
    r[17] = np.nan
    rows.append(r)
    with np.errstate(over="ignore"):
        check_quant(np.array(rows).astype(np.float32), dt)


def test_quantise_ties_swept():
    """Rows whose largest value is 127 times a power of two hold a tie at every odd half: all go to even."""
    print("case int8 quant ties", flush=True)
    n = np.arange(-253, 254, 2, dtype=np.float32)       # odd multiples of a half step
    x = np.zeros((40, 256), np.float32)
    for i in range(40):
        x[i, :254] = n / 2 * np.float32(2.0) ** (i - 20)
        x[i, 254] = 127 * np.float32(2.0) ** (i - 20)
    for dt in (torch.bfloat16, torch.float32):
        check_quant(x, dt)


def test_quantise_many_short_rows():
    """More rows than one dimension of a grid takes (2^32 threads at a wavefront a row), and 2^31 elements."""
    print("case int8 quant rows", flush=True)
    rows = (1 << 26) + 9
    x = torch.arange(32, device="cuda").to(torch.bfloat16).repeat(rows, 1)
    x[-3:, 0] = torch.tensor([40.0, 50.0, -60.0], device="cuda")
    q, s = int8_quantize(x)
    torch.cuda.synchronize()
    for at in (slice(0, 5), slice((1 << 24) - 2, (1 << 24) + 3), slice(rows - 12, rows)):
        rq, rs = quant_ref(x[at].float().cpu().numpy())
        assert np.array_equal(s[at].cpu().numpy(), rs) and np.array_equal(q[at].cpu().numpy(), rq)
    changed = int((s != s[0]).sum()), int((q != q[0]).any(1).sum())
    assert changed == (3, 3)


# ------------------------------------------------------------------------------------------------ product

def matmul_ref(q, s, w, ws, offsets, dt, M, N):
    y = np.full((M, N), np.nan, np.float32)
    groups = [(0, 0, M)] if offsets is None else [(g, offsets[g], offsets[g + 1]) for g in range(len(w))]
    for g, a, b in groups:
        W, S = (w, ws) if offsets is None else (w[g], ws[g])
        acc = np.rint(q[a:b].astype(np.float64) @ W.astype(np.float64).T)      # exact: below 2^53
        y[a:b] = acc.astype(np.float32) * (s[a:b, None] * S[None, :])
    return torch.from_numpy(y).to(dt)


def run_matmul(M, N, K, dt, offsets=None, seed=0, lo=-127):
    rng = np.random.default_rng(seed)
    G = 1 if offsets is None else len(offsets) - 1
    q = rng.integers(lo, 128, (M, K), dtype=np.int8)
    w = rng.integers(lo, 128, (G, N, K), dtype=np.int8)
    s = np.exp(rng.standard_normal(M)).astype(np.float32)
    ws = np.exp(rng.standard_normal((G, N))).astype(np.float32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to("cuda")
    if offsets is None:
        w, ws = w[0], ws[0]
    y = torch.full((M, N), float("nan"), dtype=dt, device="cuda")
    off = None if offsets is None else dev(np.asarray(offsets, np.int32))
    int8_matmul(dev(q), dev(s), dev(w), dev(ws), offsets=off, y=y)
    torch.cuda.synchronize()
    ref = matmul_ref(q, s, w, ws, offsets, dt, M, N)
    got = y.cpu()
    if not torch.equal(got.view(torch.uint8), ref.view(torch.uint8)):
        same = (got == ref) | (torch.isnan(got) & torch.isnan(ref))
        assert same.all(), (int((~same).sum()), torch.nonzero(~same)[:5].tolist())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 2048, 768), (3, 17, 80), (16, 100, 2048), (17, 33, 112), (33, 256, 64),
                                   (64, 777, 1104), (64, 16, 4096), (65, 1, 16), (65, 256, 128), (100, 300, 144),
                                   (16, 9000, 272), (33, 8192, 128), (64, 4100, 80), (256, 256, 256), (257, 264, 2048), (700, 1000, 400), (1300, 2048, 768)])
def test_product_bit_exact(M, N, K, dt):
    print("case int8 product", M, N, K, dt, flush=True)
    run_matmul(M, N, K, dt, seed=M + N + K)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("offsets,N,K", [
    ([0, 5], 40, 64),
    ([0, 0, 3, 3, 20, 64], 100, 272),                   # empty groups, a group of 44 rows
    ([2, 9, 30, 50], 64, 128),                          # rows before and behind the groups
    ([0, 1, 2, 3, 300, 301, 301, 900], 257, 208),
    ([0, 256, 512, 513, 1024, 1025], 256, 768),         # groups that end on a tile and one row past it
    ([0, 0, 0], 128, 64),                               # nothing at all
    ([7, 7, 200, 200, 500], 512, 384),
    (list(range(0, 513)), 48, 96),                      # 512 groups of one row
], ids=["one", "empty", "behind", "uneven", "tiles", "nothing", "wide", "512"])
def test_grouped_product_bit_exact(offsets, N, K, dt):
    M = max(offsets[-1] + 13, 20)                       # rows behind the last group stay NaN
    if offsets[-1] == 64:
        M = 64
    print("case int8 grouped", offsets[:9], N, K, dt, flush=True)
    run_matmul(M, N, K, dt, offsets=offsets, seed=len(offsets) + N)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("M,N,K,offsets", [(6300, 2104, 144, None), (6300, 2104, 400, [3, 3, 1000, 1100, 3660, 6271]),
                                           (20000, 520, 64, [0, 128, 257, 19900])], ids=["plain", "groups", "short"])
def test_large_product_bit_exact(M, N, K, offsets, dt):
    """Enough tiles for the 256 x 256 engine: ends inside a tile, tiles of up to 128 rows, one to four K-tiles."""
    print("case int8 large tiles", M, N, K, offsets, dt, flush=True)
    run_matmul(M, N, K, dt, offsets=offsets, seed=M)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
def test_product_into_an_odd_address(dt):
    print("case int8 odd address", dt, flush=True)
    for M, N, K in ((20, 40, 64), (300, 128, 144), (6300, 2104, 32)):
        rng = np.random.default_rng(M)
        q, w = (torch.from_numpy(rng.integers(-127, 128, s, dtype=np.int8)).cuda() for s in ((M, K), (N, K)))
        s, ws = torch.rand(M + 1, device="cuda")[1:], torch.rand(N + 3, device="cuda")[3:]
        room = torch.full((M * N + 9,), float("nan"), dtype=dt, device="cuda")
        int8_matmul(q, s, w, ws, y=room[1:1 + M * N].view(M, N))
        want = int8_matmul(q, s, w, ws, dtype=dt)
        torch.cuda.synchronize()
        assert torch.equal(room[1:1 + M * N].view(M, N), want), M
        assert torch.isnan(room[0]) and torch.isnan(room[1 + M * N:]).all(), M


def test_many_groups_of_many_channels():
    """512 groups of 2^17 channels over 60 rows: more workgroups than one dimension of a grid takes."""
    print("case int8 channels", flush=True)
    M, N, K, G = 60, 1 << 17, 16, 512
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-127, 128, (G, N, K), dtype=torch.int8, device="cuda", generator=g)
    s, ws = torch.rand(M, device="cuda", generator=g), torch.rand(G, N, device="cuda", generator=g)
    off = [0] * 200 + [31] * 312 + [60]
    y = int8_matmul(q, s, w, ws, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    for a, b, e in ((0, 31, 199), (31, 60, 511)):
        ref = (q[a:b].double() @ w[e].double().T).float() * (s[a:b, None] * ws[e])
        assert torch.equal(y[a:b], ref.to(torch.bfloat16))


def test_offsets_outside_the_rows_are_clamped():
    print("case int8 offsets clamp", flush=True)
    for M in (40, 200):
        rng = np.random.default_rng(M)
        q = torch.from_numpy(rng.integers(-127, 128, (M, 64), dtype=np.int8)).cuda()
        w = torch.from_numpy(rng.integers(-127, 128, (3, 32, 64), dtype=np.int8)).cuda()
        s, ws = torch.ones(M, device="cuda"), torch.ones(3, 32, device="cuda")
        a = int8_matmul(q, s, w, ws, offsets=torch.tensor([-9, 10, 30, M + 1000], dtype=torch.int32, device="cuda"))
        b = int8_matmul(q, s, w, ws, offsets=torch.tensor([0, 10, 30, M], dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(a, b)


def test_product_of_the_largest_bytes():
    """K at its limit with every byte 127: the sum is 131072 * 127^2, just below 2^31."""
    print("case int8 largest sums", flush=True)
    for M in (5, 70):
        run_matmul(M, 20, 131072, torch.float32, seed=1, lo=127)


def test_nan_rows_reach_their_own_outputs():
    print("case int8 nan rows", flush=True)
    for M in (20, 300):
        x = torch.randn(M, 256, device="cuda")
        w, ws = int8_quantize(torch.randn(64, 256, device="cuda"))
        x[3, 5], x[M - 1, 0] = float("nan"), float("-inf")
        y = int8_matmul(*int8_quantize(x), w, ws)
        torch.cuda.synchronize()
        bad = torch.isnan(y).all(1)
        assert bad[3] and bad[M - 1] and int(bad.sum()) == 2 and int(torch.isnan(y).any(1).sum()) == 2


def test_offsets_past_32_bits():
    """y and x of more than 2^31 elements: the last rows against the definition."""
    print("case int8 large", flush=True)
    M, N, K = 40000, 65536, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randint(-127, 128, (M, K), dtype=torch.int8, device="cuda", generator=g)
    w = torch.randint(-127, 128, (N, K), dtype=torch.int8, device="cuda", generator=g)
    s, ws = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    y = int8_matmul(q, s, w, ws)
    torch.cuda.synchronize()
    for a in (0, 20000, M - 50):
        ref = (q[a:a + 50].double() @ w.double().T).float() * (s[a:a + 50, None] * ws)
        assert torch.equal(y[a:a + 50], ref.to(torch.bfloat16)), a


# ------------------------------------------------------------------------------------------------ layer

class Case:
    def __init__(self, T, H, F, E, k, seed=501, E_local=-1, e0=0, zipf_s=0.0):
        self.cfg, self.L = inputs.custom_layer(T=T, H=H, F=F, E=E, k=k, seed=seed, E_local=E_local, e0=e0, zipf_s=zipf_s)
        L = self.L
        self.x, self.lg = to_dev(L["x"], torch.bfloat16), to_dev(L["logits"], torch.float32)
        self.w = [int8_quantize(to_dev(L[n], torch.bfloat16)) for n in ("wg", "wu", "wd")]
        self.wn = [(q.cpu().numpy().astype(np.float64), s.cpu().numpy().astype(np.float64)) for q, s in self.w]
        self.wr_np = inputs.router_weight(self.cfg)
        self.wr = to_dev(self.wr_np, torch.bfloat16)
        self.layer = Int8Layer(T, H, F, E, k, self.cfg.el, e0)
        self.layer.ws.fill_(0xFF)
        self.y = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, **kw):
        return self.layer.forward(self.x, self.lg, *self.w, self.y, **kw)

    def ref(self, logits=None):
        c = self.cfg
        r = oracle.route(self.L["logits"] if logits is None else logits, c.k, c.e0, c.el)
        x = self.L["x"].astype(np.float64)
        D = np.maximum(np.abs(x).max(1), float(FLOOR))
        xq, xs = np.rint(127 * x / D[:, None]), D / 127
        y = np.zeros_like(x)
        (wg, sg), (wu, su), (wd, sd) = self.wn
        for e in range(c.el):
            p = r["perm"][r["offsets"][e]:r["offsets"][e + 1]]
            if not len(p):
                continue
            t, wt = p // c.k, r["w"].reshape(-1)[p]
            a = (xq[t] @ wg[e].T) * xs[t, None] * sg[e]
            b = (xq[t] @ wu[e].T) * xs[t, None] * su[e]
            h = wt[:, None] * a / (1 + np.exp(-a)) * b
            Dh = np.maximum(np.abs(h).max(1), float(FLOOR))
            y[t] += (np.rint(127 * h / Dh[:, None]) @ wd[e].T) * (Dh / 127)[:, None] * sd[e]
        return y

    def check(self, y, ref):
        tol = (1 if self.cfg.T <= 64 else 2) * 2.0 ** -8 + 1e-3
        got = y.float().cpu().numpy()
        assert np.isfinite(got).all()
        err = oracle.rel_frobenius(got, ref)
        assert err <= tol, err
        n = np.linalg.norm(ref, axis=1)
        d = np.linalg.norm(got - ref, axis=1)
        assert (d <= 3 * tol * n).all(), int(np.argmax(d - 3 * tol * n))


LAYERS = [
    dict(T=1, H=256, F=128, E=1, k=1),
    dict(T=1, H=2048, F=768, E=128, k=8),
    dict(T=5, H=512, F=384, E=40, k=3),
    dict(T=17, H=768, F=128, E=6, k=6),
    dict(T=33, H=256, F=640, E=3, k=3),
    dict(T=64, H=512, F=256, E=9, k=9),
    dict(T=64, H=256, F=128, E=512, k=32, E_local=511, e0=1),
    dict(T=31, H=512, F=256, E=24, k=4, E_local=5, e0=19),
    dict(T=65, H=256, F=128, E=4, k=2),
    dict(T=100, H=512, F=256, E=64, k=6, zipf_s=2.5),
    dict(T=257, H=768, F=384, E=8, k=8),
    dict(T=300, H=256, F=128, E=300, k=20),
    dict(T=333, H=1024, F=640, E=16, k=4, E_local=4, e0=8),
    dict(T=700, H=2048, F=768, E=10, k=1),
    dict(T=1500, H=512, F=256, E=12, k=3, zipf_s=1.1),
    dict(T=2100, H=256, F=1024, E=8, k=4),              # the 256 x 256 engine for the gate/up products
    dict(T=4, H=512, F=256, E=4, k=4),                  # h quantised by the down kernel, four tokens an expert
    dict(T=2, H=2048, F=768, E=128, k=8),               # and by a launch of its own
    dict(T=8, H=512, F=384, E=5, k=5),                  # few tokens: 5 to 8 an expert, rows of h that end in half
    dict(T=12, H=2048, F=384, E=3, k=3),                # 256 bytes; 9 to 16 an expert
    dict(T=16, H=4096, F=128, E=20, k=9),
    dict(T=40, H=4096, F=640, E=24, k=6, zipf_s=1.1),
]


def name(c):
    return "-".join(f"{k}{v}" for k, v in c.items())


@pytest.mark.parametrize("c", LAYERS, ids=name)
def test_layer_matches_float64(c):
    print("case int8 layer", c, flush=True)
    k = Case(**c)
    y = k.run()
    torch.cuda.synchronize()
    k.check(y, k.ref())
    first = y.clone()
    k.layer.ws.fill_(0x55)
    y.fill_(float("nan"))
    k.run()
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("c", [
    dict(T=33, H=512, F=256, E=12, k=6),
    dict(T=65, H=256, F=128, E=4, k=2),
    dict(T=100, H=512, F=256, E=64, k=6, zipf_s=2.5),
    dict(T=300, H=256, F=128, E=300, k=20),
    dict(T=333, H=1024, F=640, E=16, k=4, E_local=4, e0=8),
    dict(T=2100, H=256, F=1024, E=8, k=4),              # the 256 x 256 engine, gate/up and down
], ids=name)
def test_layer_is_rounded_once(c):
    """Every token's y is off by half a bf16 step and fp32's accuracy, on both sides of 64 tokens. A byte of h within
    its fp32 error (2^-21 of a value of 20 steps on average) of a tie may go the other way: 2e-5 of the up to 4096
    bytes of a token, so fewer than one token in ten, are off by more."""
    print("case int8 layer accuracy", c, flush=True)
    k = Case(**c)
    y = k.run()
    torch.cuda.synchronize()
    off = excess(y.float().cpu().numpy(), k.ref())
    print("tokens past the bar", float((off > BAR).mean()), "largest", float(off.max()), flush=True)
    assert (off <= BAR).mean() >= 0.9


def test_one_formula_on_both_sides_of_64_tokens():
    """A token's h has the same bytes in a call of 64 tokens and in one of 96. Gate values of about -30, where an
    approximate exponential is off by 30 times 2^-24, and rows of h of one magnitude, most of whose bytes are large: 16384
    bytes a token, of which such an error moves one in 4e4. A moved byte shifts the token's whole row; without one the rows
    differ in the order of fp32 sums, about 1e-6 of a row's rms, which changes the rounding of one output in 10^3."""
    print("case int8 one formula", flush=True)
    T, H, F, E, k = 96, 1024, 2048, 8, 8
    g = torch.Generator(device="cuda").manual_seed(12)

    def randn(*s):
        return torch.randn(*s, device="cuda", generator=g)

    x = (1 + 0.05 * randn(T, H)).bfloat16()
    wg = -30.0 / H + 0.3 * randn(E, F, H) / H ** 0.5
    wu = 3.0 / H + 0.3 * randn(E, F, H) / H ** 0.5
    w = [int8_quantize(v) for v in (wg, wu, randn(E, H, F) / F ** 0.5)]
    lg = 0.1 * randn(T, E)
    few = Int8Layer(64, H, F, E, k).forward(x[:64], lg[:64], *w)
    many = Int8Layer(T, H, F, E, k).forward(x, lg, *w)[:64]
    torch.cuda.synchronize()
    differ = (few != many).float().mean(1)
    print("most differing outputs of a token", float(differ.max()), "tokens", int((differ > 0.02).sum()), flush=True)
    assert torch.isfinite(few).all() and (few != 0).any(1).all()
    assert float(differ.max()) <= 0.02


@pytest.mark.parametrize("H,F", [(2048, 128), (256, 2048)])
def test_layer_past_32_bits(H, F):
    """More than 2^31 elements of the pairs' outputs, or of h: the first and last tokens are those of a small call
    (each token's arithmetic is its own, and the tiles' sums are exact)."""
    print("case int8 large layer", H, F, flush=True)
    T, E, k = 140000, 8, 8
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    lg = torch.randn(T, E, device="cuda", generator=g)
    w = [int8_quantize(torch.randn(E, a, b, device="cuda", generator=g) / b ** 0.5) for a, b in ((F, H), (F, H), (H, F))]
    y = Int8Layer(T, H, F, E, k).forward(x, lg, *w)
    small = Int8Layer(100, H, F, E, k)
    for a in (0, T // 2, T - 100):
        assert torch.equal(small.forward(x[a:a + 100], lg[a:a + 100], *w), y[a:a + 100]), a


@pytest.mark.parametrize("c", [c for c in LAYERS if c["T"] <= 64 or c["E"] <= 256][::2]
                         + [dict(T=90, H=256, F=128, E=40, k=12)], ids=name)
def test_layer_with_the_router(c):
    print("case int8 layer router", c, flush=True)
    k = Case(**c)
    y, lg = k.layer.forward_router(k.x, k.wr, *k.w, k.y)
    torch.cuda.synchronize()
    got = lg.cpu().numpy()
    assert oracle.rel_frobenius(got, oracle.router_forward(k.L["x"], k.wr_np)) <= 1e-5
    k.check(y, k.ref(logits=got))


def test_layer_share_without_tokens_is_zero():
    print("case int8 layer empty share", flush=True)
    for T in (6, 90):
        k = Case(T=T, H=256, F=128, E=8, k=2, E_local=2, e0=6)
        k.lg[:, 6:] = -torch.finfo(torch.float32).max
        y = k.run()
        torch.cuda.synchronize()
        assert torch.count_nonzero(y) == 0 and torch.isfinite(y).all()


@pytest.mark.parametrize("T", [5, 90])
def test_layer_masked_logits(T):
    print("case int8 layer masked", T, flush=True)
    k = Case(T=T, H=256, F=128, E=6, k=3)
    y0 = k.run().clone()
    k.lg[1, 2:] = float("-inf")                         # two experts left for three slots
    k.lg[3] = float("-inf")
    k.lg[4, 3] = float("nan")
    y = k.run()
    torch.cuda.synchronize()
    rest = [t for t in range(T) if t not in (1, 3, 4)]
    assert torch.isnan(y[3:5]).all() and torch.isfinite(y[1]).all() and torch.equal(y[rest], y0[rest])


def test_layer_nan_token_stays_alone():
    print("case int8 layer nan token", flush=True)
    for T in (20, 150):
        k = Case(T=T, H=256, F=128, E=4, k=4)
        y0 = k.run().clone()
        k.x[7, 3], k.x[11, 0] = float("nan"), float("inf")
        y1 = k.run()
        torch.cuda.synchronize()
        rest = [t for t in range(T) if t not in (7, 11)]
        assert torch.isnan(y1[[7, 11]]).all() and torch.equal(y0[rest], y1[rest])


@pytest.mark.parametrize("router", [False, True])
def test_layer_nan_token_with_more_than_eight_slots(router):
    """Logits that are NaN choose experts whose weights are NaN: the token's y is NaN, never zeros."""
    print("case int8 layer nan top-12", router, flush=True)
    for T in (20, 90):
        k = Case(T=T, H=256, F=128, E=40, k=12)

        def run():
            return k.layer.forward_router(k.x, k.wr, *k.w, k.y)[0].clone() if router else k.run().clone()

        y0 = run()
        if router:
            k.x[7, 3], k.x[11, 0] = float("nan"), float("inf")
        else:
            k.lg[7] = float("nan")
            k.lg[11, 5] = float("nan")
        y1 = run()
        torch.cuda.synchronize()
        rest = [t for t in range(T) if t not in (7, 11)]
        assert torch.isnan(y1[[7, 11]]).all() and torch.equal(y0[rest], y1[rest]), T


def test_prompt_then_tokens_with_one_set_of_weights():
    """A server's path: weights quantised once, a prompt through the grouped products, its rows again as few
    tokens, and the composition of the public calls (quantise, grouped product by the routing's offsets)."""
    print("case int8 serving run", flush=True)
    T, H, F, E, k = 130, 512, 256, 16, 4
    c = Case(T=T, H=H, F=F, E=E, k=k)
    y = c.run().float()
    out, t = [], 0
    for n in (64, 1, 33, 32):
        out.append(Int8Layer(n, H, F, E, k).forward(c.x[t:t + n], c.lg[t:t + n], *c.w))
        t += n
    few = torch.cat(out).float()
    # the same by hand
    r = oracle.route(c.L["logits"], k)
    tok = torch.from_numpy(r["perm"] // k).cuda()
    off = torch.from_numpy(np.asarray(r["offsets"], np.int32)).cuda()
    wt = torch.from_numpy(r["w"].reshape(-1)[r["perm"]].astype(np.float32)).cuda()
    xq, xs = int8_quantize(c.x)
    a = int8_matmul(xq[tok], xs[tok], *c.w[0], offsets=off, dtype=torch.float32)
    b = int8_matmul(xq[tok], xs[tok], *c.w[1], offsets=off, dtype=torch.float32)
    o = int8_matmul(*int8_quantize(wt[:, None] * torch.nn.functional.silu(a) * b), *c.w[2], offsets=off,
                    dtype=torch.float32)
    hand = torch.zeros(T, H, device="cuda").index_add_(0, tok, o)
    torch.cuda.synchronize()
    ref = c.ref()
    c.check(y, ref)
    for v in (few, hand):
        assert oracle.rel_frobenius(v.cpu().numpy(), ref) <= 2.0 ** -8 + 1e-3
    # against the bf16 weights: the bytes of weights and rows are off by half of 1/127 of the row's largest
    bf = FewTokenLayer(64, H, F, E, k).forward(c.x[:64], c.lg[:64], *(to_dev(c.L[n], torch.bfloat16) for n in ("wg", "wu", "wd")))
    assert oracle.rel_frobenius(few[:64].cpu().numpy(), bf.float().cpu().numpy()) <= 0.05


def test_new_outputs_on_another_stream():
    """Outputs made for calls on a side stream are no memory that the current stream still writes."""
    print("case int8 side stream", flush=True)
    x = torch.randn(512, 1024, device="cuda")
    want = int8_quantize(x)
    y = int8_matmul(*want, *want, dtype=torch.float32)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        old = [torch.empty_like(t) for t in (*want, y)]
        torch.cuda._sleep(20_000_000)
        [t.fill_(5) for t in old]
        del old                                         # freed while the current stream has yet to write them
        for stream in (side, side.cuda_stream, side):
            got = int8_quantize(x, stream=stream)
            z = int8_matmul(*got, *got, dtype=torch.float32, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(z, y)


def stream_of(t):
    """The handle of the stream from whose memory t was made."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("no segment")


def test_new_outputs_come_from_the_given_streams_memory():
    """A stream given as an object or as a handle, the null stream's handle 0 among them."""
    print("case int8 output streams", flush=True)
    x = torch.randn(48, 256, device="cuda")
    q, s = int8_quantize(x)
    k, few = Case(T=5, H=256, F=128, E=8, k=2), FewTokenLayer(5, 256, 128, 8, 2)
    w = [to_dev(k.L[n], torch.bfloat16) for n in ("wg", "wu", "wd")]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for current in (torch.cuda.default_stream(), side):
        for given in (0, torch.cuda.default_stream(), side.cuda_stream, side, None):
            want = given if isinstance(given, int) else (given or current).cuda_stream
            with torch.cuda.stream(current):
                new = [*int8_quantize(x, stream=given), int8_matmul(q, s, q, s, stream=given),
                       k.layer.forward(k.x, k.lg, *k.w, stream=given),
                       *k.layer.forward_router(k.x, k.wr, *k.w, stream=given),
                       few.forward(k.x, k.lg, *w, stream=given), *few.forward_router(k.x, k.wr, *w, stream=given)]
            torch.cuda.synchronize()
            assert [stream_of(t) for t in new] == [want] * len(new), (current, given)


@pytest.mark.parametrize("T,router", [(9, False), (9, True), (40, False), (130, False), (130, True)])
def test_layer_graph_replays(T, router):
    print("case int8 graph", T, router, flush=True)
    k = Case(T=T, H=512, F=256, E=16, k=4)
    lg = torch.empty(T, 16, device="cuda")

    def step():
        if router:
            k.layer.forward_router(k.x, k.wr, *k.w, k.y, lg)
        else:
            k.run()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x0 = k.x.clone()
    for r in range(4):
        k.x.copy_(x0 * (1 + r))
        step()
        torch.cuda.synchronize()
        want = k.y.clone()
        k.y.fill_(float("nan"))
        k.layer.ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want.view(torch.uint8), k.y.view(torch.uint8)), r


def test_two_threads_on_their_own_streams():
    print("case int8 threads", flush=True)
    cases = [Case(T=11, H=512, F=256, E=16, k=4, seed=51), Case(T=200, H=256, F=384, E=8, k=2, seed=52)]
    want = [c.run().clone() for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        torch.cuda.set_device(0)
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                cases[i].y.fill_(float("nan"))
                cases[i].run()
                if not torch.equal(cases[i].y, want[i]):
                    bad.append(i)

    th = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in th]
    [t.join() for t in th]
    assert not bad
