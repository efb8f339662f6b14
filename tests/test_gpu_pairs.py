"""Pairs sorted by expert, dispatch, combine and their gradients on the GPU, against plain implementations in 64 bits."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_32_amd import binding as b
from mixture_experts_layer_32_amd.layer import (GradNorm, MoELayer, combine, combine_backward, dispatch, int8_matmul,
                                                int8_quantize, sort_pairs)

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24                                   # half a step of fp32
DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "int8": torch.int8}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def ref_sort(idx, El, e0):
    """offsets, perm, pair_pos by Python's stable sort."""
    e = idx.reshape(-1).tolist()
    here = sorted((v, q) for q, v in enumerate(e) if e0 <= v < e0 + El)
    perm = [q for _, q in here] + [-1] * (len(e) - len(here))
    pos = [-1] * len(e)
    for i, (_, q) in enumerate(here):
        pos[q] = i
    counts = np.bincount([v - e0 for v, _ in here], minlength=El) if here else np.zeros(El, np.int64)
    return np.concatenate([[0], np.cumsum(counts)]), np.array(perm), np.array(pos).reshape(idx.shape)


def check_sort(idx, El, e0):
    got = sort_pairs(idx.to(DEV), El, e0)
    for g, r in zip(got, ref_sort(idx, El, e0)):
        np.testing.assert_array_equal(g.cpu().numpy(), r)
    return got


def choose(T, k, E, seed, drop=0.0, zipf=0.0):
    g = gen(seed)
    p = torch.arange(1, E + 1).double() ** -zipf
    idx = torch.multinomial(p.expand(T, E).contiguous(), k, generator=g) if k <= E else torch.randint(0, E, (T, k), generator=g)
    idx = torch.where(torch.rand(T, k, generator=g) < drop, -1, idx)
    return idx.int()


@pytest.mark.parametrize("T,k,E,El,e0", [
    (1, 1, 1, 1, 0), (1, 8, 128, 128, 0), (8, 8, 128, 128, 0), (63, 3, 5, 5, 0), (64, 1, 512, 512, 0),
    (511, 8, 64, 64, 0), (512, 8, 128, 16, 16), (513, 8, 128, 128, 0), (4096, 1, 512, 512, 0), (4097, 1, 7, 3, 2),
    (2731, 3, 100, 100, 0), (1333, 6, 128, 16, 112), (16384, 8, 128, 128, 0), (300, 32, 512, 512, 0), (32768, 8, 40, 40, 0), (32769, 8, 300, 200, 50),
    (70001, 2, 300, 257, 43),
])
def test_sort(T, k, E, El, e0):
    check_sort(choose(T, k, E, T + k, zipf=1.0 if T % 2 else 0.0), El, e0)


@pytest.mark.parametrize("T,k", [(5, 2), (700, 9), (9000, 4)])
def test_sort_drops_strangers_and_repeats(T, k):
    g = gen(T)
    idx = torch.randint(-3, 12, (T, k), generator=g).int()           # repeats inside a token, experts outside 2..8
    idx[0, 0], idx[-1, -1] = -2 ** 31, 2 ** 31 - 1
    check_sort(idx, 7, 2)
    check_sort(torch.full((T, k), -1).int(), 7, 2)                   # nothing has a position
    check_sort(torch.full((T, k), 8).int(), 7, 2)                    # everything in the last expert


@pytest.mark.parametrize("T,k,E,El,e0", [(70001, 8, 9, 5, 2), (140001, 8, 300, 300, 0), (262145, 8, 600, 512, 50),
                                         (1048577, 1, 3, 3, 0)])
def test_sort_of_many_blocks(T, k, E, El, e0):
    """More than 256 and 512 blocks of 2048 pairs, whose counts are scanned 256 at a time; experts drawn unevenly, with
    dropped ones."""
    r = np.random.default_rng(T)
    idx = (E * r.random((T, k)) ** 2).astype(np.int32)
    idx[r.random((T, k)) < 0.1] = -1
    flat = idx.reshape(-1).astype(np.int64) - e0
    flat = np.where((flat >= 0) & (flat < El), flat, El)
    order = np.argsort(flat, kind="stable")
    P = int((flat < El).sum())
    pos = np.empty_like(order)
    pos[order] = np.arange(T * k)
    offsets, perm, pair_pos = (t.cpu().numpy() for t in sort_pairs(torch.from_numpy(idx).to(DEV), El, e0))
    np.testing.assert_array_equal(offsets, np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=El + 1)[:El])]))
    np.testing.assert_array_equal(perm[:P], order[:P])
    assert (perm[P:] == -1).all()
    np.testing.assert_array_equal(pair_pos.reshape(-1), np.where(flat < El, pos, -1))


def test_sort_agrees_with_the_layer():
    T, E, k = 1000, 32, 4
    layer = MoELayer(T, 256, 128, E, k, "bf16", E_local=12, expert_offset=8)
    layer.route(torch.randn(T, E, generator=gen(1)).to(DEV))
    p = layer.pairs()
    offsets, perm, pair_pos = sort_pairs(p["idx"], 12, 8)
    P = int(offsets[-1])
    assert torch.equal(offsets, p["offsets"]) and torch.equal(pair_pos, p["pair_pos"])
    assert torch.equal(perm[:P], p["perm"][:P]) and bool((perm[P:] == -1).all())
    r = layer.routing()
    for n in ("idx", "weight", "offsets"):
        assert torch.equal(r[n], p[n].cpu())


# (T, k, H): single tokens, row lengths around the pieces that a wave takes, odd ones, many slots
SHAPES = [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (5, 4, 1001), (64, 8, 256), (33, 3, 1024), (17, 6, 1032), (9, 32, 264),
          (130, 8, 2048), (21, 5, 4100), (6, 2, 16392), (300, 2, 30)]


def layout(T, k, seed, drop=0.25, spare=3):
    """pair_pos of a random choice with dropped pairs, tokens without any, and rows that no pair stands at."""
    idx = choose(T, k, max(k, 6), seed, drop)
    idx[T // 2] = -1
    _, _, pos = ref_sort(idx, max(k, 6), 0)
    n = int((pos >= 0).sum()) + spare
    return idx, torch.from_numpy(pos).int(), n


def offset_view(t, elements):
    """t's values behind an address that is `elements` elements off a 16-byte boundary."""
    buf = torch.zeros(t.numel() + 16, dtype=t.dtype, device=t.device)
    v = buf[elements:elements + t.numel()].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", ["bf16", "fp32", "int8"])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_dispatch(T, k, H, dtype):
    _, pos, n = layout(T, k, T + H)
    x = (torch.randn(T, H, generator=gen(H)) * 30).to(DT[dtype])
    for off in (0, 1):
        rows = offset_view(torch.full((n, H), 77, dtype=DT[dtype], device=DEV), off)
        dispatch(offset_view(x.to(DEV), off), pos.to(DEV), rows=rows)
        want = torch.full((n, H), 77, dtype=DT[dtype])
        t, j = torch.nonzero(pos >= 0, as_tuple=True)
        want[pos[t, j].long()] = x[t]
        assert torch.equal(rows.cpu(), want)


def test_dispatch_makes_rows_for_every_pair():
    pos = torch.tensor([[1, 0], [3, 2]], dtype=torch.int32, device=DEV)
    x = torch.randn(2, 48, device=DEV)
    assert torch.equal(dispatch(x, pos), x[[0, 0, 1, 1]])


def close(got, ref, dtype, err):
    """|got - ref| within half a step of dtype at the larger of the two and err (an array: what the fp32 arithmetic
    ahead of the rounding may be off by); 2^-133 is half the smallest bf16 and above half the smallest fp32."""
    got, ref, err = (torch.as_tensor(t).double().cpu() for t in (got, ref, err))
    bound = HALF[dtype] * torch.maximum(got.abs(), ref.abs()) + err + 2.0 ** -133
    bad = ~((got - ref).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, by up to {((got - ref).abs() / bound).max():.3g} bounds"


@pytest.mark.parametrize("rows_type,dtype", [("bf16", "bf16"), ("fp32", "fp32"), ("fp32", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("T,k,H", SHAPES)
def test_combine_and_gradients(T, k, H, rows_type, dtype):
    idx, pos, n = layout(T, k, 3 * T + H)
    g = gen(T * H)
    rt, dt = DT[rows_type], DT[dtype]
    rows, dy = torch.randn(n, H, generator=g).to(rt), torch.randn(T, H, generator=g).to(dt)
    w = torch.softmax(torch.randn(T, k, generator=g), -1)
    here = (pos >= 0).double()
    r = rows.double()[pos.clamp(min=0).long()] * here[..., None]              # [T, k, H]
    E = max(k, 6)
    for off in (0, 1):
        d_rows, d_dy, d_pos = offset_view(rows.to(DEV), off), offset_view(dy.to(DEV), off), pos.to(DEV)
        # y: k fused multiply-adds, each off by U of the running sum
        for wt, wd in ((w.to(DEV), w.double()), (None, torch.ones(T, k).double())):
            y = offset_view(torch.full((T, H), 9.0, dtype=dt, device=DEV), off)
            combine(d_rows, d_pos, wt, y=y)
            terms = wd[..., None] * r
            close(y, terms.sum(1), dt, k * U * terms.abs().sum(1))
        assert torch.equal(combine(d_rows, d_pos, w.to(DEV), dtype=dt), combine(d_rows, d_pos, w.to(DEV), y=y))
        # gradients
        drows = offset_view(torch.full((n, H), 5.0, dtype=rt, device=DEV), off)
        out = combine_backward(d_dy, d_rows, w.to(DEV), d_pos, idx=idx.to(DEV), E_total=E, drows=drows)
        want = torch.full((n, H), 5.0).double()
        t, j = torch.nonzero(pos >= 0, as_tuple=True)
        want[pos[t, j].long()] = w.double()[t, j][:, None] * dy.double()[t]
        # one product in fp32, then the rounding to the rows' type
        close(out[0], want, rt, U * want.abs())
        # dot: a lane adds at most H/64 + 16 products in fp32, then six additions across the wave
        prod = dy.double()[:, None] * r
        dw, edw = prod.sum(-1), (H / 64 + 24) * U * prod.abs().sum(-1)
        close(out[1], dw, torch.float32, edw)
        assert bool((out[1].cpu()[pos < 0] == 0).all())
        wd = w.double()
        m = (wd * dw).sum(-1, keepdim=True)
        dl = wd * (dw - m)
        mag = (wd * dw.abs()).sum(-1, keepdim=True)
        edl = wd * (edw + (wd * edw).sum(-1, keepdim=True) + (k + 4) * U * (dw.abs() + mag))
        full, efull = torch.zeros(T, E).double(), torch.zeros(T, E).double()
        t, j = torch.nonzero(idx >= 0, as_tuple=True)
        full[t, idx[t, j].long()], efull[t, idx[t, j].long()] = dl[t, j], edl[t, j]
        close(out[2], full, torch.float32, efull)
        two = combine_backward(d_dy, d_rows, w.to(DEV), d_pos, drows=torch.empty_like(drows))
        assert len(two) == 2 and torch.equal(two[1], out[1])


def test_a_token_may_name_an_expert_twice():
    idx = torch.tensor([[2, 2, 0, -1], [7, 1, 7, 7]], dtype=torch.int32, device=DEV)      # 7 is beyond E_total below
    _, _, pos = sort_pairs(idx, 8)
    g = gen(0)
    rows, dy = torch.randn(8, 64, generator=g).to(DEV), torch.randn(2, 64, generator=g).to(DEV)
    w = torch.softmax(torch.randn(2, 4, generator=g), -1).to(DEV)
    _, dw, dl = combine_backward(dy, rows, w, pos, idx=idx, E_total=7)
    each = w * (dw - (w * dw).sum(-1, keepdim=True))
    want = torch.zeros(2, 7, device=DEV)
    want[0, 2], want[0, 0], want[1, 1] = each[0, 0] + each[0, 1], each[0, 2], each[1, 1]
    assert dw[0, 3] == 0
    torch.testing.assert_close(dl, want, rtol=1e-6, atol=1e-6)      # four fp32 roundings of values of order 1


def test_masked_rows_are_neither_read_nor_written():
    """Values that are not finite at no pair's position, and positions beyond the rows, change nothing."""
    pos = torch.tensor([[0, -1, 900], [2, 1, -7], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    rows = torch.randn(5, 40, device=DEV)
    rows[3:] = float("nan")
    w = torch.rand(3, 3, device=DEV)
    y = combine(rows, pos, w)
    assert torch.equal(y[2], torch.zeros(40, device=DEV))
    want = torch.stack([w[0, 0] * rows[0], torch.addcmul(w[1, 0] * rows[2], w[1, 1], rows[1])])
    torch.testing.assert_close(y[:2], want, rtol=2 ** -22, atol=2 ** -22)
    drows, dw = combine_backward(torch.ones(3, 40, device=DEV), rows, w, pos, drows=torch.full_like(rows, 4.0))
    assert bool((drows[3:] == 4).all()) and bool((dw[pos < 0] == 0).all()) and dw[0, 2] == 0
    rows[1] = float("inf")                       # one pair's values reach its own token alone
    y = combine(rows, pos, w)
    assert bool(torch.isinf(y[1]).all()) and bool(torch.isfinite(y[[0, 2]]).all())


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H", [40, 1024, 5000])
def test_weights_of_masked_slots_reach_nothing_else(H, value):
    """A slot without a position adds nothing to y; its weight reaches no gradient but its own logit's."""
    idx = torch.tensor([[0, -1, 2], [3, 1, 4], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([[0, -1, 3], [2, 1, -1], [-1, -1, -1]], dtype=torch.int32, device=DEV)
    g = gen(H)
    rows, dy = torch.randn(4, H, generator=g).to(DEV), torch.randn(3, H, generator=g).to(DEV)
    w = torch.rand(3, 3, generator=g).to(DEV)
    bad = torch.where(pos < 0, value, w)

    def gradients(weight):
        return combine_backward(dy, rows, weight, pos, idx=idx, E_total=6, drows=torch.zeros_like(rows))
    assert torch.equal(combine(rows, pos, bad), combine(rows, pos, w))
    (drows, dw, dl), (want_rows, want_dw, want_dl) = gradients(bad), gradients(w)
    assert torch.equal(drows, want_rows) and torch.equal(dw, want_dw)
    own = torch.zeros(3, 6, dtype=torch.bool, device=DEV)
    own[1, 4] = True                               # the masked slot with an expert: weight (0 - sum)
    assert torch.equal(dl[~own], want_dl[~own]) and not bool(torch.isfinite(dl[own]).any())


def test_gradients_against_differences():
    """Of rows and weights, in which y is linear, the differences are exact but for rounding; of the logits, through the
    softmax over the chosen experts, central differences in 64 bits."""
    T, k, E, H = 40, 4, 9, 96
    g = gen(5)
    idx = choose(T, k, E, 5)
    _, _, pos = sort_pairs(idx.to(DEV), E)
    logits = torch.randn(T, E, generator=g).double()
    rows, dy = torch.randn(T * k, H, generator=g), torch.randn(T, H, generator=g)
    chosen = torch.gather(logits, 1, idx.long())
    w = torch.softmax(chosen, -1).float()
    dr, dw, dl = combine_backward(dy.to(DEV), rows.to(DEV), w.to(DEV), pos, idx=idx.to(DEV), E_total=E)

    def f(rows, weight):
        r = rows[pos.cpu().long()]
        return (dy.double()[:, None] * weight[..., None] * r).sum().item()
    R, W = rows.double(), w.double()
    v, u = torch.randn(T * k, H, generator=g).double(), torch.randn(T, k, generator=g).double()
    # each gradient element is off by some U of its terms; their sums over all elements by less than 1e-4 of the terms' size
    for got, want, size in (((dr.cpu().double() * v).sum().item(), f(R + v, W) - f(R, W), (dr.cpu().double() * v).abs().sum()),
                            ((dw.cpu().double() * u).sum().item(), f(R, W + u) - f(R, W), (dw.cpu().double() * u).abs().sum())):
        assert abs(got - want) <= 1e-5 * float(size)
    h = 1e-4
    for t in range(0, T, 7):
        for e in range(E):
            d = torch.zeros(T, E).double()
            d[t, e] = h
            hi, lo = (f(R, torch.softmax(torch.gather(logits + s * d, 1, idx.long()), -1)) for s in (1, -1))
            # h^2 / 6 of a third derivative below 6 |dw|, the cancellation in 64 bits, and fp32's rounding of dw and w
            size = float((w[t] * dw[t].cpu().abs()).sum())
            assert abs((hi - lo) / (2 * h) - float(dl[t, e])) <= 1e-5 * size + 1e-6


def test_rows_beyond_two_to_the_31_elements():
    """Positions whose elements pass 32 bits: 140000 rows of 16384 bf16, two slots a token."""
    T, k, H = 70000, 2, 16384
    idx = torch.zeros(T, k, dtype=torch.int32, device=DEV)
    idx[:, 1] = 1
    _, _, pos = sort_pairs(idx, 2)
    x = torch.randn(T, H, device=DEV, dtype=torch.bfloat16)
    rows = dispatch(x, pos)
    assert rows.numel() > 2 ** 31
    assert torch.equal(rows[T - 1], x[T - 1]) and torch.equal(rows[T:], x) and torch.equal(rows[:T], x)
    w = torch.full((T, k), 0.5, device=DEV)
    assert torch.equal(combine(rows, pos, w), x)
    drows, dw = combine_backward(x, rows, w, pos)
    assert torch.equal(drows[T:], x * 0.5) and torch.equal(dw[:, 0], dw[:, 1])
    assert bool((dw > 0).all())


def test_results_do_not_change_from_call_to_call():
    idx, pos, n = layout(500, 8, 3)
    rows, dy, w = torch.randn(n, 1000, device=DEV), torch.randn(500, 1000, device=DEV), torch.rand(500, 8, device=DEV)
    first = None
    for _ in range(3):
        out = [combine(rows, pos.to(DEV), w), *combine_backward(dy, rows, w, pos.to(DEV), idx=idx.to(DEV), E_total=8,
                                                                 drows=torch.zeros_like(rows))]
        first = first or out
        assert all(torch.equal(a, c) for a, c in zip(first, out))


@pytest.mark.parametrize("T", [16, 2000])
def test_captured_and_replayed(T):
    """sort, dispatch, combine and the gradients in one graph, replayed with new inputs between eager work."""
    k, E, H = 8, 64, 512
    g = gen(T)
    idx = choose(T, k, E, 1).to(DEV)
    x, w, dy = torch.randn(T, H, device=DEV), torch.rand(T, k, device=DEV), torch.randn(T, H, device=DEV)

    def work():
        offsets, perm, pos = sort_pairs(idx, 40, 8)
        rows = dispatch(x, pos, rows=torch.zeros(T * k, H, device=DEV))
        return [offsets, perm, pos, rows, combine(rows, pos, w),
                *combine_backward(dy, rows, w, pos, idx=idx, E_total=E, drows=torch.zeros_like(rows))]
    work()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        idx.copy_(choose(T, k, E, 10 + i, drop=0.1))
        x.normal_()
        torch.cuda.synchronize()
        graph.replay()
        want = work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(out, want))


@pytest.mark.parametrize("kind", ["object", "handle", "null"])
def test_on_a_given_stream(kind):
    T, k, E, H = 3000, 4, 16, 256
    idx = choose(T, k, E, 2).to(DEV)
    x = torch.randn(T, H, device=DEV)
    want_pos = sort_pairs(idx, E)[2]
    want = combine(dispatch(x, want_pos), want_pos)
    side = torch.cuda.Stream()
    s = {"object": side, "handle": side.cuda_stream, "null": 0}[kind]
    torch.cuda.synchronize()
    pos = sort_pairs(idx, E, stream=s)[2]
    y = combine(dispatch(x, pos, stream=s), pos, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(pos, want_pos) and torch.equal(y, want)


def test_without_tokens_or_rows():
    idx = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    offsets, perm, pos = sort_pairs(idx, 5)
    assert offsets.tolist() == [0] * 6 and perm.numel() == 0 and pos.shape == (0, 3)
    x, w = torch.zeros((0, 8), device=DEV), torch.zeros((0, 3), device=DEV)
    rows = dispatch(x, pos)
    assert rows.shape == (0, 8) and combine(rows, pos, w).shape == (0, 8)
    out = combine_backward(x, rows, w, pos, idx=idx, E_total=4)
    assert [tuple(t.shape) for t in out] == [(0, 8), (0, 3), (0, 4)]
    # tokens, none of whose pairs has a row
    idx = torch.full((5, 3), 9, dtype=torch.int32, device=DEV)
    offsets, perm, pos = sort_pairs(idx, 5)
    assert offsets.tolist() == [0] * 6 and bool((perm == -1).all()) and bool((pos == -1).all())
    x, w, rows = torch.ones((5, 8), device=DEV), torch.ones((5, 3), device=DEV), torch.zeros((0, 8), device=DEV)
    dispatch(x, pos, rows=rows)
    assert torch.equal(combine(rows, pos, w), torch.zeros_like(x))
    drows, dw, dl = combine_backward(x, rows, w, pos, idx=idx, E_total=10)
    assert drows.shape == (0, 8) and bool((dw == 0).all()) and bool((dl == 0).all())


def test_wrong_tensors_are_refused():
    idx = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    x = torch.zeros(4, 16, device=DEV)
    w = torch.zeros(4, 2, device=DEV)
    for call in (lambda: sort_pairs(idx.long(), 4), lambda: sort_pairs(idx.t(), 4), lambda: sort_pairs(idx[0], 4),
                 lambda: dispatch(x.double(), idx), lambda: dispatch(x, idx[:3]), lambda: dispatch(x, idx.long()),
                 lambda: dispatch(x[:, ::2], idx), lambda: dispatch(x, idx, rows=torch.zeros(8, 15, device=DEV)),
                 lambda: dispatch(x, idx, rows=torch.zeros(8, 16, device=DEV, dtype=torch.bfloat16)),
                 lambda: combine(x, idx, w.double()), lambda: combine(x, idx, w[:3]), lambda: combine(x.to(torch.int8), idx),
                 lambda: combine(x, idx, dtype=torch.float16), lambda: combine(x, idx, y=torch.zeros(4, 15, device=DEV)),
                 lambda: combine_backward(x, x, w, idx, idx=idx), lambda: combine_backward(x, x, w, idx, E_total=4),
                 lambda: combine_backward(x[:3], x, w, idx), lambda: combine_backward(x, x, None, idx),
                 lambda: combine_backward(x, x, w, idx, drows=x[:3]), lambda: sort_pairs(idx, 2 ** 32 + 4),
                 lambda: sort_pairs(idx, 4, 2 ** 32),
                 lambda: combine_backward(x, x, w, idx, idx=idx, E_total=2 ** 32 + 128),
                 lambda: combine_backward(x, x, w, idx, idx=idx, E_total=0)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sort_pairs(idx, 0), lambda: sort_pairs(idx, 4, -1),
                 lambda: dispatch(x[:, :0].contiguous(), idx)):
        with pytest.raises(b.MoEError):
            call()


def test_the_8_bit_layer_taken_apart():
    """route, quantised rows and their scales dispatched, grouped 8-bit products and combine, against moe_fwd on the
    weights that the bytes stand for."""
    T, H, F, E, k = 300, 256, 128, 8, 2
    g = gen(11)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    wg, wu, wd = (torch.randn(s, generator=g).to(DEV) / s[-1] ** 0.5 for s in ((E, F, H), (E, F, H), (E, H, F)))
    route = MoELayer(T, H, F, E, k, "bf16")
    route.route(logits)
    p = route.pairs()
    (qg, sg), (qu, su), (qd, sd) = (int8_quantize(w) for w in (wg, wu, wd))
    q, s = int8_quantize(x)
    rows, scales = dispatch(q, p["pair_pos"]), dispatch(s[:, None], p["pair_pos"])[:, 0].contiguous()
    a, c = (int8_matmul(rows, scales, w, ws, offsets=p["offsets"], dtype=torch.float32) for w, ws in ((qg, sg), (qu, su)))
    hq, hs = int8_quantize(torch.nn.functional.silu(a) * c)
    y = combine(int8_matmul(hq, hs, qd, sd, offsets=p["offsets"], dtype=torch.float32), p["pair_pos"], p["weight"])
    layer = MoELayer(T, H, F, E, k, "fp32")
    want = layer.forward(x.float(), logits, *(v.float() * u[..., None] for v, u in ((qg, sg), (qu, su), (qd, sd))))
    # a row's rounding to bytes: 1/254 of its largest value at most, 0.3 of that in the mean square; twice (x and h)
    err = float((y - want).norm() / want.norm())
    assert err <= 2e-2


def test_a_training_step_with_experts_of_its_own():
    """route, dispatch, the caller's experts in torch, combine; the gradients all the way back, against moe_bwd of the
    layer with the same experts; then the norm over all gradients and their scaling, against torch's."""
    T, H, F, E, k = 200, 256, 128, 6, 3
    g = gen(12)
    x, dy = torch.randn(T, H, generator=g).to(DEV), torch.randn(T, H, generator=g).to(DEV)
    logits = torch.randn(T, E, generator=g).to(DEV)
    wg, wu, wd = (torch.randn(s, generator=g).to(DEV) / s[-1] ** 0.5 for s in ((E, F, H), (E, F, H), (E, H, F)))
    layer = MoELayer(T, H, F, E, k, "fp32")
    y_ref = layer.forward(x, logits, wg, wu, wd)
    ref = layer.backward(dy, x, wg, wu, wd)
    p = {n: t.clone() for n, t in layer.pairs().items()}
    rows = dispatch(x, p["pair_pos"]).requires_grad_()
    params = [w.clone().requires_grad_() for w in (wg, wu, wd)]
    bounds, parts = p["offsets"].tolist(), []
    for e in range(E):
        r = rows[bounds[e]:bounds[e + 1]]
        parts.append((torch.nn.functional.silu(r @ params[0][e].T) * (r @ params[1][e].T)) @ params[2][e].T)
    out = torch.cat(parts)
    y = combine(out.detach(), p["pair_pos"], p["weight"])
    dout, dweight, dlogits = combine_backward(dy, out.detach(), p["weight"], p["pair_pos"], idx=p["idx"], E_total=E)
    grads = torch.autograd.grad(out, [rows, *params], dout)
    dx = combine(grads[0], p["pair_pos"])

    def err(a, r):
        return float((a - r).norm() / r.norm())
    # both sides in fp32 throughout: sums of up to 256 terms, three deep
    for a, r in ((y, y_ref), (dx, ref["dx"]), (dlogits, ref["dlogits"]), (grads[1], ref["dw_gate"]),
                 (grads[2], ref["dw_up"]), (grads[3], ref["dw_down"])):
        assert err(a, r) <= 2e-5
    mine = [ref[n] for n in ("dw_gate", "dw_up", "dw_down")]
    theirs = [torch.nn.Parameter(w) for w in (wg, wu, wd)]
    for t, m in zip(theirs, mine):
        t.grad = m.clone()
    want = torch.nn.utils.clip_grad_norm_(theirs, 0.5)
    norm = GradNorm(mine).clip(0.5)
    assert abs(float(norm) / float(want) - 1) <= 1e-5
    for t, m in zip(theirs, mine):
        torch.testing.assert_close(m, t.grad, rtol=2e-5, atol=0)
