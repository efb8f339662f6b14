"""Products with 4-bit weights on the GPU, against plain implementations in 64 bits."""
import pytest
import torch

from mixture_experts_layer_32_amd import binding as b
from mixture_experts_layer_32_amd.layer import MoELayer, combine, dispatch, int4_matmul, int4_pack, int4_quantize

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def unpack(q, s, N, K):
    """(values, scales) [.., N, K] that the tiles hold, by the layout that the header gives."""
    group = 128 // s.shape[-1]
    n, k = torch.arange(N, device=DEV)[:, None], torch.arange(K, device=DEV)[None]
    c, i, h, j = n % 64 // 4, k % 128 // 32, k % 32 // 8, k % 8
    flags = q[..., -16:].contiguous().view(torch.int32)[..., 0]              # [.., N / 64]
    words = q[..., :-16].contiguous().view(torch.int32).long() & 0xffffffff
    words = words.unflatten(-1, (4, -1, 256))                                # [.., N / 64, 4, K / 128, 256]
    w = words[..., n // 64, n % 4, k // 128, (16 * h + c) * 4 + i]
    m = (w >> torch.where(j < 4, 8 * j, 8 * (j - 4) + 4)) & 7
    sign = (w >> torch.where(j < 4, 8 * j + 7, (8 * (j - 4) + 11) % 32)) & 1
    v = torch.where(sign == 1, torch.where(m == 0, -8, -m), m)
    for r in range(flags.shape[-1]):                                         # a word says whether 64 channels hold a -8
        assert torch.equal(flags[..., r] != 0, (v[..., 64 * r:64 * r + 64, :] == -8).flatten(-2).any(-1))
    return v, s[..., n // 64, k // 128, n % 64, (k % 128) // group]


def quantised(w, group):
    """The definition: D / 7 in fp32, at least 2^-126, as bf16; the nearest whole number to the quotient in 64 bits."""
    g = w.double().unflatten(-1, (-1, group))
    D = w.float().unflatten(-1, (-1, group)).abs().amax(-1)
    s = (D / 7).clamp(min=2.0 ** -126).to(torch.bfloat16)
    bad = ~torch.isfinite(D)
    q = (g / s.double()[..., None]).round().clamp(-7, 7)
    q = torch.where(bad[..., None], 0.0, q).flatten(-2)
    return q.long(), torch.where(bad, float("nan"), s.float()).to(torch.bfloat16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape,group", [((1, 32), 32), ((16, 128), 128), ((17, 160), 32), ((5, 192), 64), ((33, 1024), 128),
                                         ((3, 20, 96), 32), ((4, 16, 256), 64), ((2, 7, 384), 128)])
def test_quantize(shape, group, dtype):
    g = gen(sum(shape))
    w = (torch.randn(shape, generator=g, device=DEV) * torch.exp(3 * torch.randn((*shape[:-1], 1), generator=g, device=DEV)))
    w = w.to(dtype)
    w[..., 0, :group] = 0
    # ties, from both sides: the largest value 7 or 14 gives s = 1 or 2, halves lie between two whole numbers
    if shape[-2] > 2:
        w[..., 1, :8] = torch.tensor([7, 0.5, 1.5, 2.5, -0.5, -1.5, -3.5, 6.5], device=DEV).to(dtype)
        w[..., 1, 8:group] = 0
        w[..., 2, :4] = torch.tensor([-14, 1, 3, 5], device=DEV).to(dtype)
        w[..., 2, 4:group] = 0
    q, s = int4_quantize(w, group)
    v, sc = unpack(q, s, shape[-2], shape[-1])
    want_v, want_s = quantised(w, group)
    assert torch.equal(v, want_v)
    assert torch.equal(sc, want_s.repeat_interleave(group, -1))
    p, ps = int4_pack(want_v.to(torch.int8), want_s)
    assert torch.equal(p, q) and torch.equal(ps, s)


def test_quantize_values_that_are_not_finite_and_padding():
    w = torch.randn(3, 64, device=DEV)
    w[0, 5], w[1, 40] = float("nan"), -float("inf")
    w[2, :32] = 1e-42
    w[2, 32:] = 3e38
    q, s = int4_quantize(w, 32)
    v, sc = unpack(q, s, 64, 128)
    assert bool(sc[0, :32].isnan().all()) and bool((v[0, :32] == 0).all()) and bool(sc[1, 32:64].isnan().all())
    want_v, want_s = quantised(w, 32)
    assert torch.equal(v[:3, :64], want_v)
    assert bool((v[3:] == 0).all()) and bool((v[:, 64:] == 0).all())              # padding
    assert bool((sc[3:] == 0).all()) and bool((sc[:, 64:] == 0).all())


def test_pack_takes_the_nearer_of_the_bounds():
    v = torch.arange(-128, 128, device=DEV).to(torch.int8).view(1, 256)
    q, s = int4_pack(v, torch.ones(1, 8, dtype=torch.bfloat16, device=DEV))
    assert torch.equal(unpack(q, s, 1, 256)[0], v.long().clamp(-8, 7))


@pytest.mark.parametrize("G,N,K", [(1, 70, 4096), (3, 130, 2080), (512, 64, 256)])
def test_one_number_of_minus_8_is_found_wherever_it_is(G, N, K):
    g = gen(K)
    s = torch.ones((G, N, K // 32), dtype=torch.bfloat16, device=DEV)
    for at in [(0, 0, 0), (G - 1, N - 1, K - 1), (G // 2, N // 2, K // 2 + 5), (0, N - 1, 600 % K), None]:
        v = torch.randint(-7, 8, (G, N, K), generator=g, device=DEV).to(torch.int8)
        if at:
            v[at] = -8
        q, sc = int4_pack(v, s)                    # (unpack compares the words with what the numbers are)
        assert torch.equal(unpack(q, sc, N, K)[0], v.long())


def rand_weight(shape, group, g, exact=False, low=-8):
    v = torch.randint(low, 8, shape, generator=g, device=DEV).to(torch.int8)
    s = torch.rand((*shape[:-1], shape[-1] // group), generator=g, device=DEV) + 0.5
    s = torch.exp2((4 * s).floor() - 4) if exact else s / shape[-1] ** 0.5
    return v, s.to(torch.bfloat16)


def real(v, s, group):
    return v.double() * s.double().repeat_interleave(group, -1)


def offsets_of(M, G, g, skew=1.0, lead=0, tail=0):
    p = torch.arange(1, G + 1, device=DEV).double() ** -skew
    n = torch.bincount(torch.multinomial(p, M - lead - tail, replacement=True, generator=g), minlength=G) if M > lead + tail else torch.zeros(G, dtype=torch.long, device=DEV)
    return torch.cat([n.new_zeros(1), n.cumsum(0)]).int() + lead


def bound(x, v, s, group):
    """What fp32 sums may be off by: in a group each input adds up to 8 |x|, in at most `group` additions; the groups'
    sums are then added in K / group fused steps (K / 64 of half groups at most), and 16 across the waves."""
    K = x.shape[-1]
    size = x.double().abs() @ s.double().abs().repeat_interleave(group, -1).transpose(-1, -2)
    return (group + K / min(group, 64) + 16) * U * 8 * size


# (M, N, K): one row to several tiles of rows, odd everything, one group of inputs, long rows
SHAPES = [(1, 1, 32), (1, 16, 128), (1, 1536, 4096), (2, 33, 96), (7, 777, 1120), (16, 100, 512), (17, 48, 640), (31, 130, 1024),
          (33, 64, 2048), (64, 256, 1024), (65, 40, 320), (128, 128, 128), (200, 300, 544), (257, 513, 1056), (1000, 96, 768),
          (3, 16, 16384), (700, 1024, 2048), (40, 4096, 512), (200, 2112, 256), (520, 4160, 192), (2100, 4100, 224), (5000, 2056, 160),
          (300, 1300, 96), (330, 1500, 384), (9000, 1801, 96), (8500, 2048, 160),
          (1000, 4100, 160), (1000, 4101, 352)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(M, N, K, group, out):
    K = -(-K // group) * group
    g = gen(M * N + K)
    # whole numbers and scales that are powers of two: every sum is exact in fp32, so that y is exactly rounded
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(torch.bfloat16)
    for low in (-8, -7):                           # with and without the number that takes more steps to unpack
        v, s = rand_weight((N, K), group, g, exact=True, low=low)
        if low == -8 and N > 64:
            v[64:128].clamp_(min=-7)               # one run of 64 channels without it among others
        want = x.double() @ real(v, s, group).T
        assert torch.equal(int4_matmul(x, *int4_pack(v, s), N=N, dtype=out), want.to(out))
    # real values
    v, s = rand_weight((N, K), group, g)
    x = (torch.randn(M, K, generator=g, device=DEV) * torch.exp(torch.randn(M, 1, generator=g, device=DEV))).to(torch.bfloat16)
    y = int4_matmul(x, *int4_pack(v, s), N=N, dtype=out).double()
    want = x.double() @ real(v, s, group).T
    assert bool(((y - want).abs() <= HALF[out] * torch.maximum(y.abs(), want.abs()) + bound(x, v, s, group)).all())


# (M, G, N, K, skew, rows ahead of the first group, rows behind the last)
GROUPS = [(1, 1, 16, 32, 0, 0, 0), (1, 8, 40, 256, 0, 0, 0), (8, 16, 768, 512, 0, 0, 0), (64, 128, 192, 1024, 0, 0, 0), (64, 16, 64, 128, 2, 0, 0),
          (50, 7, 33, 160, 1, 3, 5), (300, 5, 100, 416, 1, 11, 30), (1117, 9, 777, 1120, 2, 0, 0), (2000, 130, 64, 256, 1, 0, 7),
          (900, 2, 257, 352, 4, 1, 1), (40, 512, 16, 64, 0, 0, 0), (6, 4, 32, 128, 0, 3, 3),
          (3000, 20, 513, 256, 0, 2, 1), (9000, 24, 640, 192, 1, 0, 9), (700, 200, 130, 128, 0, 0, 0),
          (14000, 20, 1100, 160, 0.5, 3, 5), (800, 12, 900, 640, 0, 0, 4),
          (3000, 100, 900, 416, 0.5, 2, 3), (9000, 24, 1100, 96, 1, 0, 9)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,G,N,K,skew,lead,tail", GROUPS)
def test_grouped(M, G, N, K, skew, lead, tail, group):
    K = -(-K // group) * group
    g = gen(M + G + N)
    off = offsets_of(M, G, g, skew, lead, tail)
    v, s = rand_weight((G, N, K), group, g, exact=True)
    v[::2].clamp_(min=-7)                          # every other weight without a -8
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(torch.bfloat16)
    for out in (torch.bfloat16, torch.float32):
        want = torch.full((M, N), 6.0, dtype=out, device=DEV)
        y = want.clone()
        for e, (a, z) in enumerate(zip(off.tolist(), off.tolist()[1:])):
            want[a:z] = (x[a:z].double() @ real(v[e], s[e], group).T).to(out)
        int4_matmul(x, *int4_pack(v, s), offsets=off, y=y)
        assert torch.equal(y, want)


def test_offsets_outside_the_rows():
    """Offsets below 0 and beyond M are taken as the nearer of the two."""
    g = gen(3)
    v, s = rand_weight((4, 32, 64), 32, g, exact=True)
    x = torch.randint(-4, 5, (100, 64), generator=g, device=DEV).to(torch.bfloat16)
    w = int4_pack(v, s)
    good = int4_matmul(x, *w, N=32, offsets=torch.tensor([0, 0, 90, 100, 100], dtype=torch.int32, device=DEV))
    far = torch.tensor([-70, -5, 90, 1000, 2 ** 31 - 1], dtype=torch.int32, device=DEV)
    assert torch.equal(int4_matmul(x, *w, N=32, offsets=far), good)
    y = torch.full((100, 32), 2.0, device=DEV)
    int4_matmul(x, *w, offsets=torch.tensor([100, 100, 100, 100, 100], dtype=torch.int32, device=DEV), y=y)
    assert bool((y == 2).all())


@pytest.mark.parametrize("M", [1, 5, 70, 600])
def test_values_that_are_not_finite(M):
    g = gen(M)
    v, s = rand_weight((48, 256), 64, g, exact=True)
    x = torch.randint(-4, 5, (M, 256), generator=g, device=DEV).to(torch.bfloat16)
    want = (x.double() @ real(v, s, 64).T).float()
    x[M // 2, 77] = float("nan")
    bad = torch.zeros(M, dtype=torch.bool, device=DEV)
    bad[M // 2] = True
    if M > 2:
        x[M - 1, 3], bad[M - 1] = float("inf"), True
    y = int4_matmul(x, *int4_pack(v, s), N=48, dtype=torch.float32)
    assert torch.equal(y[~bad], want[~bad]) and not bool(torch.isfinite(y[bad]).any())
    s[5, 1] = float("nan")                         # a group's scale: its channel alone
    y = int4_matmul(x, *int4_pack(v, s), N=48, dtype=torch.float32)
    keep = torch.arange(48, device=DEV) != 5
    assert bool(y[:, 5].isnan().all()) and torch.equal(y[~bad][:, keep], want[~bad][:, keep])


def test_large_and_small_values():
    """Rows near bf16's largest and smallest values, whose sums still lie within fp32."""
    g = gen(8)
    v, s = rand_weight((32, 128), 32, g, exact=True)
    x = torch.randint(-4, 5, (3, 128), generator=g, device=DEV).float()
    x = (x * torch.tensor([[2.0 ** 110], [2.0 ** -110], [1.0]], device=DEV)).to(torch.bfloat16)
    assert torch.equal(int4_matmul(x, *int4_pack(v, s), N=32, dtype=torch.float32), (x.double() @ real(v, s, 32).T).float())


def test_more_than_two_to_the_31_numbers():
    """A weight of 2^31 numbers and more in 16 groups, and an output beyond 2^31 elements."""
    G, N, K = 16, 8208, 16384
    v = torch.zeros((G, N, K), dtype=torch.int8, device=DEV)
    v[:, :, 5] = 3
    v[-1, -1] = 1
    s = torch.ones((G, N, K // 128), dtype=torch.bfloat16, device=DEV)
    w = int4_pack(v, s)
    assert v.numel() > 2 ** 31
    del v
    x = torch.zeros((G, K), dtype=torch.bfloat16, device=DEV)
    x[:, 5], x[-1, -1] = 1, 2
    y = int4_matmul(x, *w, offsets=torch.arange(G + 1, dtype=torch.int32, device=DEV), N=N, dtype=torch.float32)
    want = torch.full((G, N), 3.0, device=DEV)
    want[-1, -1] = 3.0                             # 1 * 1 + 2 * 1
    assert torch.equal(y, want)
    del w, y
    M, N, K = 70000, 32768, 32
    w = int4_pack(torch.full((N, K), 2, dtype=torch.int8, device=DEV), torch.ones((N, 1), dtype=torch.bfloat16, device=DEV))
    x = torch.ones((M, K), dtype=torch.bfloat16, device=DEV)
    x[-1] = 3
    y = int4_matmul(x, *w)
    assert y.numel() > 2 ** 31 and bool((y[:-1] == 64).all()) and bool((y[-1] == 192).all())


def test_weights_of_2_to_the_22_runs_of_64_channels():
    """More of them than a launch takes workgroups of 1024 threads along one dimension."""
    G, N, K = 256, 1 << 20, 32
    g = gen(12)
    assert G * N // 64 == 1 << 22
    v = torch.randint(-7, 8, (G, N, K), generator=g, device=DEV, dtype=torch.int8)
    at = [0, 127, 128, 255]                        # groups on both sides of the first 2^21 runs, and the last
    for e in at:
        v[e, 5::640, 7] = -8
    s = torch.ones((G, N, 1), dtype=torch.bfloat16, device=DEV)
    q, sc = int4_pack(v, s)
    x = torch.randint(-4, 5, (G, K), generator=g, device=DEV).to(torch.bfloat16)
    y = int4_matmul(x, q, sc, offsets=torch.arange(G + 1, dtype=torch.int32, device=DEV), dtype=torch.float32)
    for e in range(G):
        assert torch.equal(y[e], v[e].float() @ x[e].float())        # whole numbers below 2^24: exact
    del q, sc, y, s
    w = v.to(torch.bfloat16)
    del v
    q, sc = int4_quantize(w, 32)
    for e in at:
        one_q, one_s = int4_quantize(w[e], 32)
        assert torch.equal(q[e], one_q) and torch.equal(sc[e], one_s)


def test_rows_that_pass_4_gib():
    """x of more than 2^32 bytes in one group: rows of the first tiles, of the last and of one between, among zeros."""
    M, N, K = 2 ** 14 + 3, 64, 2 ** 17
    g = gen(11)
    v, s = rand_weight((N, K), 128, g, exact=True)
    q, sc = int4_pack(v, s)
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    at = torch.tensor([0, 2, 3, 63, 64, 255, 8191, M - 4, M - 1], device=DEV)
    rows = torch.randint(-1, 2, (len(at), K), generator=g, device=DEV).to(torch.bfloat16)
    x[at] = rows
    y = int4_matmul(x, q, sc, dtype=torch.float32)
    # whole quarters below 2^17 * 8 * 2: exact in fp32
    want = torch.zeros((M, N), device=DEV)
    want[at] = (rows.double() @ real(v, s, 128).T).float()
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [4, 300])
def test_captured_and_replayed(M):
    g = gen(M)
    v, s = rand_weight((6, 80, 256), 64, g, exact=True)
    w = int4_pack(v, s)
    x = torch.zeros((M, 256), dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(7, dtype=torch.int32, device=DEV)
    y = torch.zeros((M, 80), device=DEV)
    int4_matmul(x, *w, offsets=off, y=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        int4_matmul(x, *w, offsets=off, y=y)
    for i in range(4):
        x.copy_(torch.randint(-4, 5, (M, 256), generator=g, device=DEV))
        off.copy_(offsets_of(M, 6, g))
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(y, int4_matmul(x, *w, N=80, offsets=off, dtype=torch.float32))


@pytest.mark.parametrize("kind", ["object", "handle", "null"])
def test_on_a_given_stream(kind):
    g = gen(4)
    v, s = rand_weight((96, 256), 64, g)
    x = torch.randn(40, 256, generator=g, device=DEV).to(torch.bfloat16)
    want = int4_matmul(x, *int4_pack(v, s), N=96)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    h = {"object": side, "handle": side.cuda_stream, "null": 0}[kind]
    y = int4_matmul(x, *int4_pack(v, s, stream=h), N=96, stream=h)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


def test_odd_addresses_of_y():
    g = gen(6)
    v, s = rand_weight((50, 128), 32, g, exact=True)
    for M in (3, 300):
        x = torch.randint(-4, 5, (M, 128), generator=g, device=DEV).to(torch.bfloat16)
        for out in (torch.bfloat16, torch.float32):
            buf = torch.full((M * 50 + 9,), 4.0, dtype=out, device=DEV)
            y = buf[1:1 + M * 50].view(M, 50)
            int4_matmul(x, *int4_pack(v, s), y=y)
            assert torch.equal(y, (x.double() @ real(v, s, 32).T).to(out))
            assert bool((buf[:1] == 4).all()) and bool((buf[1 + M * 50:] == 4).all())


# shapes for each of the kernels that the library chooses from (on 256 CUs): few rows by 1 and by 4 tiles a wave (5 and
# more rows by one tile the other form of the first), 64 x 64 tiles with two groups of waves and with one, 64 x 128,
# 128 x 128 and 256 x 128 tiles
KERNELS = [pytest.param(3, 100, id="rows1_few"), pytest.param(60, 100, id="rows1"), pytest.param(12, 20000, id="rows4"),
           pytest.param(330, 1500, id="deep2"), pytest.param(520, 2080, id="deep1"), pytest.param(2100, 2080, id="wide"),
           pytest.param(2100, 4100, id="tile128"), pytest.param(8500, 2048, id="tile256")]


GROUPED = [pytest.param(40, 9, 72, id="rows1"), pytest.param(100, 9, 4096, id="rows4"), pytest.param(700, 9, 1000, id="deep2"),
           pytest.param(1000, 9, 1300, id="deep1"), pytest.param(3000, 100, 900, id="wide"),
           pytest.param(3000, 20, 2080, id="tile128"), pytest.param(9000, 5, 2048, id="tile256")]
# inputs of 5 and more times 128, an odd and an even number of them, whole ones and 32, 64 and 96 more; groups
LONG = [(640, 128), (1120, 32), (1152, 64), (1184, 32), (1216, 64), (2048, 32), (2048, 64), (2048, 128)]


@pytest.mark.parametrize("K,group", LONG)
@pytest.mark.parametrize("M,N", KERNELS)
def test_long_rows_on_every_kernel(M, N, K, group):
    g = gen(M + K)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(torch.bfloat16)
    for low in (-8, -7):
        v, s = rand_weight((N, K), group, g, exact=True, low=low)
        want = x.double() @ real(v, s, group).T     # quarters below 2^19: exact in fp32
        assert torch.equal(int4_matmul(x, *int4_pack(v, s), N=N, dtype=torch.float32), want.float())


@pytest.mark.parametrize("K,group", [(1120, 32), (1216, 64), (2048, 128)])
@pytest.mark.parametrize("M,N", KERNELS)
def test_real_values_in_long_rows_on_every_kernel(M, N, K, group):
    g = gen(M * K)
    v, s = rand_weight((N, K), group, g)
    x = (torch.randn(M, K, generator=g, device=DEV) * torch.exp(torch.randn(M, 1, generator=g, device=DEV))).to(torch.bfloat16)
    want = x.double() @ real(v, s, group).T
    for out in (torch.bfloat16, torch.float32):
        y = int4_matmul(x, *int4_pack(v, s), N=N, dtype=out).double()
        assert bool(((y - want).abs() <= HALF[out] * torch.maximum(y.abs(), want.abs()) + bound(x, v, s, group)).all())


@pytest.mark.parametrize("K,group", [(640, 128), (1120, 32), (1216, 64), (2048, 128)])
@pytest.mark.parametrize("M,G,N", GROUPED)
def test_long_rows_in_groups(M, G, N, K, group):
    g = gen(M + K)
    off = offsets_of(M, G, g, 0.3, 3, 4)
    v, s = rand_weight((G, N, K), group, g, exact=True)
    v[::2].clamp_(min=-7)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(torch.bfloat16)
    want = torch.full((M, N), 6.0, device=DEV)
    y = want.clone()
    bounds = off.tolist()
    for e in range(G):
        want[bounds[e]:bounds[e + 1]] = (x[bounds[e]:bounds[e + 1]].double() @ real(v[e], s[e], group).T).float()
    int4_matmul(x, *int4_pack(v, s), offsets=off, y=y)
    assert torch.equal(y, want)


@pytest.mark.parametrize("K", [256, 352])
@pytest.mark.parametrize("M,N", KERNELS)
def test_values_that_are_not_finite_on_every_kernel(M, N, K):
    g = gen(M)
    v, s = rand_weight((N, K), 32, g, exact=True)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(torch.bfloat16)
    want = (x.double() @ real(v, s, 32).T).float()
    bad = torch.zeros(M, dtype=torch.bool, device=DEV)
    for r, k, value in ((M // 2, 77, float("nan")), (M - 1, K - 1, float("inf")), (0, 3, -float("inf"))):
        x[r, k], bad[r] = value, True
    y = int4_matmul(x, *int4_pack(v, s), N=N, dtype=torch.float32)
    assert torch.equal(y[~bad], want[~bad]) and not bool(torch.isfinite(y[bad]).any())
    s[5, 1], s[N - 1, K // 32 - 1] = float("nan"), float("inf")            # groups' scales: their channels alone
    v[N - 1, K - 32:] = 1
    x[:, K - 32:] = 1
    want = (x.double() @ real(v, torch.where(torch.isfinite(s), s, 1), 32).T).float()
    y = int4_matmul(x, *int4_pack(v, s), N=N, dtype=torch.float32)
    keep = torch.ones(N, dtype=torch.bool, device=DEV)
    keep[5] = keep[N - 1] = False
    assert bool(y[:, 5].isnan().all()) and bool(torch.isinf(y[~bad][:, N - 1]).all())
    bad[M - 1] = False                              # (that infinity stood among the last inputs)
    assert torch.equal(y[~bad][:, keep], want[~bad][:, keep])


@pytest.mark.parametrize("M,G,N", GROUPED)
def test_rows_of_other_groups_that_are_not_finite(M, G, N):
    """The rows at the groups' ends, and those outside of all groups, hold NaN: the rows beside them do not see it."""
    g = gen(M)
    K = 224
    off = offsets_of(M, G, g, 0, 3, 4)
    v, s = rand_weight((G, N, K), 32, g, exact=True)
    x = torch.randint(-4, 5, (M, K), generator=g, device=DEV).to(torch.bfloat16)
    want = torch.full((M, N), 6.0, device=DEV)
    bounds = off.tolist()
    for e in range(G):
        want[bounds[e]:bounds[e + 1]] = (x[bounds[e]:bounds[e + 1]].double() @ real(v[e], s[e], 32).T).float()
    x[:3] = float("nan")
    x[M - 4:] = float("inf")
    bad = torch.zeros(M, dtype=torch.bool, device=DEV)
    for e in range(0, G, 2):
        if bounds[e + 1] > bounds[e]:
            x[bounds[e + 1] - 1], bad[bounds[e + 1] - 1] = float("nan"), True
    y = torch.full((M, N), 6.0, device=DEV)
    int4_matmul(x, *int4_pack(v, s), offsets=off, y=y)
    assert torch.equal(y[~bad], want[~bad]) and bool(y[bad].isnan().all())


@pytest.mark.parametrize("M,G,N", GROUPED)
def test_offsets_outside_the_rows_on_every_kernel(M, G, N):
    g = gen(G)
    v, s = rand_weight((G, N, 160), 32, g, exact=True)
    w = int4_pack(v, s)
    x = torch.randint(-4, 5, (M, 160), generator=g, device=DEV).to(torch.bfloat16)
    off = offsets_of(M, G, g, 0)
    off[-2] = M                                     # the last group is empty
    good = int4_matmul(x, *w, N=N, offsets=off, dtype=torch.float32)
    far = off.clone()
    far[0], far[-2], far[-1] = -2 ** 31, M + 1, 2 ** 31 - 1
    assert torch.equal(int4_matmul(x, *w, N=N, offsets=far, dtype=torch.float32), good)
    off[:] = torch.where(torch.arange(G + 1, device=DEV) > G // 2, M, 0)     # one group has every row
    want = (x.double() @ real(v[G // 2], s[G // 2], 32).T).float()
    assert torch.equal(int4_matmul(x, *w, N=N, offsets=off, dtype=torch.float32), want)


@pytest.mark.parametrize("M,G,N", GROUPED)
def test_captured_and_replayed_on_every_kernel(M, G, N):
    g = gen(N)
    v, s = rand_weight((G, N, 384), 64, g, exact=True)
    w = int4_pack(v, s)
    x = torch.zeros((M, 384), dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(G + 1, dtype=torch.int32, device=DEV)
    y = torch.zeros((M, N), device=DEV)
    int4_matmul(x, *w, offsets=off, y=y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        int4_matmul(x, *w, offsets=off, y=y)
    for i in range(4):
        x.copy_(torch.randint(-4, 5, (M, 384), generator=g, device=DEV))
        off.copy_(offsets_of(M, G, g, 0.5 * i))
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        assert torch.equal(y, int4_matmul(x, *w, N=N, offsets=off, dtype=torch.float32))
        bounds = off.tolist()
        for e in range(G):
            want = x[bounds[e]:bounds[e + 1]].double() @ real(v[e], s[e], 64).T
            assert torch.equal(y[bounds[e]:bounds[e + 1]], want.float())


@pytest.mark.parametrize("M,N", KERNELS)
def test_odd_addresses_of_y_on_every_kernel(M, N):
    """N a multiple of 4 and y an element or two off: rows are stored element by element, or by two."""
    g = gen(N)
    v, s = rand_weight((N, 160), 32, g, exact=True)
    w = int4_pack(v, s)
    x = torch.randint(-4, 5, (M, 160), generator=g, device=DEV).to(torch.bfloat16)
    want = x.double() @ real(v, s, 32).T
    for out in (torch.bfloat16, torch.float32):
        for lead in (1, 2):
            buf = torch.full((M * N + 9,), 4.0, dtype=out, device=DEV)
            y = buf[lead:lead + M * N].view(M, N)
            int4_matmul(x, *w, y=y)
            assert torch.equal(y, want.to(out))
            assert bool((buf[:lead] == 4).all()) and bool((buf[lead + M * N:] == 4).all())


@pytest.mark.parametrize("M,N", KERNELS)
def test_on_a_given_stream_on_every_kernel(M, N):
    g = gen(M)
    v, s = rand_weight((N, 256), 64, g, exact=True)
    w = int4_pack(v, s)
    x = torch.randint(-4, 5, (M, 256), generator=g, device=DEV).to(torch.bfloat16)
    want = (x.double() @ real(v, s, 64).T).float()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = int4_matmul(x, *w, N=N, dtype=torch.float32, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("M,N", KERNELS)
def test_another_width_than_the_weights_is_seen(M, N):
    """K within the same 128 inputs cannot be told from the tensors' shapes; the tiles say it, and y is NaN."""
    g = gen(M)
    v, s = rand_weight((N, 256), 32, g, exact=True)
    x = torch.randint(-4, 5, (M, 256), generator=g, device=DEV).to(torch.bfloat16)
    whole, less = int4_pack(v, s), int4_pack(v[:, :224].contiguous(), s[:, :7].contiguous())
    narrow = x[:, :224].contiguous()
    for out in (torch.bfloat16, torch.float32):
        assert bool(int4_matmul(narrow, *whole, N=N, dtype=out).isnan().all())
        assert bool(int4_matmul(x, *less, N=N, dtype=out).isnan().all())
        assert torch.equal(int4_matmul(narrow, *less, N=N, dtype=out), (narrow.double() @ real(v[:, :224], s[:, :7], 32).T).to(out))
    quantised = int4_quantize(real(v, s, 32).float()[:, :224].contiguous(), 32)
    assert bool(int4_matmul(x, *quantised, N=N).isnan().all())
    assert bool(torch.isfinite(int4_matmul(narrow, *quantised, N=N)).all())
    for words in ((1, 1, 1), (0, 0, 0), (-1, -1, -1)):                # tiles whose words do not tell K
        q = whole[0].clone()
        q[:, -12:].view(torch.int32)[:] = torch.tensor(words, dtype=torch.int32, device=DEV)
        assert torch.equal(int4_matmul(x, q, whole[1], N=N), int4_matmul(x, *whole, N=N))


@pytest.mark.parametrize("M,G,N", [(40, 9, 70), (700, 9, 1000), (1000, 9, 1300), (3000, 100, 900), (3000, 20, 2080), (9000, 5, 2048)])
def test_another_width_in_one_group(M, G, N):
    g = gen(G)
    v, s = rand_weight((G, N, 128), 32, g, exact=True)
    q, sc = int4_pack(v, s)
    q[2] = int4_pack(v[2, :, :96].contiguous(), s[2, :, :3].contiguous())[0]
    x = torch.randint(-4, 5, (M, 128), generator=g, device=DEV).to(torch.bfloat16)
    off = offsets_of(M, G, g, 0)
    y = int4_matmul(x, q, sc, offsets=off, N=N, dtype=torch.float32)
    for e, (a, z) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        if e == 2:
            assert z > a and bool(y[a:z].isnan().all())
        else:
            assert torch.equal(y[a:z], (x[a:z].double() @ real(v[e], s[e], 32).T).float())


def test_wrong_tensors_are_refused():
    g = gen(1)
    v, s = rand_weight((32, 128), 64, g)
    q, sc = int4_pack(v, s)
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device=DEV)
    off = torch.zeros(2, dtype=torch.int32, device=DEV)
    for call in (lambda: int4_matmul(x.float(), q, sc), lambda: int4_matmul(x[0], q, sc), lambda: int4_matmul(x[:, ::2], q, sc),
                 lambda: int4_matmul(x, q[..., :4096], sc), lambda: int4_matmul(x, q, sc[..., :1]),
                 lambda: int4_matmul(x, q, sc.float()), lambda: int4_matmul(x, q, sc, offsets=off),
                 lambda: int4_matmul(x, q[None], sc[None], offsets=off.long()), lambda: int4_matmul(x, q[None], sc[None]),
                 lambda: int4_matmul(x, q, sc, N=0), lambda: int4_matmul(x, q, sc, N=65),
                 lambda: int4_matmul(x, q, sc, dtype=torch.float16),
                 lambda: int4_matmul(x, q, sc, y=torch.zeros((5, 32), device=DEV)),
                 lambda: int4_matmul(torch.zeros((4, 256), dtype=torch.bfloat16, device=DEV), q, sc),
                 lambda: int4_quantize(x, 48), lambda: int4_quantize(x.half()), lambda: int4_quantize(x[0]),
                 lambda: int4_pack(v, s.float()), lambda: int4_pack(v, s[:3]), lambda: int4_pack(v.long(), s),
                 lambda: int4_pack(v, s[:, :0])):
        with pytest.raises(ValueError):
            call()
    assert int4_matmul(x[:0], q, sc).shape == (0, 64)
    for call in (lambda: int4_matmul(x[:, :96].contiguous(), q, sc),
                 lambda: int4_quantize(torch.zeros((4, 80), device=DEV), 32)):
        with pytest.raises(b.MoEError):
            call()


@pytest.mark.parametrize("T", [1, 8, 300])
def test_the_layer_with_4_bit_weights(T):
    """route, dispatch, grouped 4-bit products with the activation between them, combine; against the layer's forward in
    fp32 on the values that the numbers stand for."""
    H, F, E, k, group = 512, 256, 16, 4, 64
    g = gen(T)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    logits = torch.randn(T, E, generator=g, device=DEV)
    ws = [torch.randn(s, generator=g, device=DEV) / s[-1] ** 0.5 for s in ((E, F, H), (E, F, H), (E, H, F))]
    route = MoELayer(T, H, F, E, k, "bf16")
    route.route(logits)
    p = route.pairs()
    (qg, sg), (qu, su), (qd, sd) = packed = [int4_quantize(w, group) for w in ws]
    rows = dispatch(x, p["pair_pos"])
    a = int4_matmul(rows, qg, sg, offsets=p["offsets"], dtype=torch.float32)
    c = int4_matmul(rows, qu, su, offsets=p["offsets"], dtype=torch.float32)
    h = (torch.nn.functional.silu(a) * c).to(torch.bfloat16)
    o = int4_matmul(h, qd, sd, offsets=p["offsets"], dtype=torch.float32)
    y = combine(o, p["pair_pos"], p["weight"], dtype=torch.bfloat16)
    vals = []
    for (q, s), w in zip(packed, ws):
        v, sc = unpack(q, s, w.shape[1], w.shape[2])
        vals.append((v * sc).float().contiguous())
    want = MoELayer(T, H, F, E, k, "fp32").forward(x.float(), logits, *vals)
    # h and y are rounded to bf16: two errors of at most 2^-8 of each value
    assert float((y.float() - want).norm() / want.norm()) <= 2 * 2.0 ** -8
