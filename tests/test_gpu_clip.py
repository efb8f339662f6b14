"""The norm over many gradients and their scaling on the GPU, against 64 bits."""
import pytest
import torch

from mixture_experts_layer_32_amd import binding as b
from mixture_experts_layer_32_amd.layer import GradNorm

pytestmark = pytest.mark.gpu
DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def make(sizes, types, seed=0, lead=0):
    """Tensors one behind the other in one buffer of each type, `lead` elements behind its start."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = [None] * len(sizes)
    for dt in (torch.bfloat16, torch.float32):
        mine = [i for i in range(len(sizes)) if types[i % len(types)] == dt]
        buf = torch.full((lead + sum(sizes[i] for i in mine) + 8,), 3.0, dtype=dt, device=DEV)
        at = lead
        for i in mine:
            out[i] = buf[at:at + sizes[i]]
            out[i].copy_(torch.randn(sizes[i], generator=g, device=DEV) * 10.0 ** (-i % 5 - 1))
            at += sizes[i]
    return out


def ref_norm(ts):
    return float(torch.stack([(t.double() ** 2).sum() for t in ts]).sum().sqrt())


BF, FP = torch.bfloat16, torch.float32
LISTS = [([1], [BF]), ([7], [FP]), ([0, 5, 0], [FP]), ([8191], [BF]), ([8192], [FP]), ([8193], [BF]), ([100003], [FP]),
         ([3, 17, 4096, 1, 0, 70001, 255, 8192, 33], [BF, FP]), (list(range(1, 330)), [FP, BF, BF]),
         ([16] * 700, [BF, FP]), ([5000003, 2, 1 << 20], [BF]), ([40000001], [FP, BF]), ([5000000] * 3 + [1000000] * 600, [BF, BF, FP])]


@pytest.mark.parametrize("lead", [0, 1, 3])
@pytest.mark.parametrize("sizes,types", LISTS)
def test_norm_and_clip(sizes, types, lead):
    ts = make(sizes, types, len(sizes), lead)
    want = ref_norm(ts)
    plan = GradNorm(ts)
    norm = plan.norm()
    assert norm.dtype == torch.float32 and norm.shape == ()
    # squares and sums in 64 bits, one rounding to fp32
    assert abs(float(norm) - want) <= 2.0 ** -24 * want * (1 + 1e-6)
    was = [t.clone() for t in ts]
    assert torch.equal(plan.clip(2 * want), norm)                      # within the bound: nothing changes
    assert all(torch.equal(a, c) for a, c in zip(ts, was))
    bound = 0.4 * want
    c = min(1.0, bound / (want + 1e-6))
    for out_types in ([BF, FP], [FP, BF, FP]):
        out = make(sizes, out_types, 9, lead)
        other = GradNorm(ts, out)
        assert torch.equal(other.clip(bound), norm)
        for t, o in zip(ts, out):
            check_scaled(t, o, c)
        assert torch.equal(other.clip(3 * want), norm)                 # within: copied
        for t, o in zip(ts, out):
            assert torch.equal(o, t.to(o.dtype))
    given = torch.full((1,), want * 2, device=DEV)
    assert plan.clip(want, norm=given) is given                        # scaled by a norm from elsewhere
    for t, o in zip(was, ts):
        check_scaled(t, o, min(1.0, want / (2 * want + 1e-6)))
    for t, o in zip(was, ts):
        o.copy_(t)
    assert torch.equal(plan.clip(bound), norm)                         # in place
    for t, o in zip(was, ts):
        check_scaled(t, o, c)


def check_scaled(t, o, c):
    """o = c t: c is off by the roundings of the norm, the sum and the quotient (3 half steps of fp32, 4 with the second
    order), the product by one, and o is rounded once more."""
    if t.numel() == 0:
        return
    want = c * t.double()
    bound = (5 * 2.0 ** -24 + HALF[o.dtype]) * (1 + 2.0 ** -7) * want.abs() + 2.0 ** -133
    assert bool(((o.double() - want).abs() <= bound).all())


def test_memory_around_the_tensors_is_left_alone():
    buf = torch.full((40000,), 2.0, dtype=torch.bfloat16, device=DEV)
    ts = [buf[1:4], buf[9:8210], buf[8211:39993]]
    GradNorm(ts).clip(1.0)
    inside = torch.zeros(40000, dtype=torch.bool, device=DEV)
    for a, z in ((1, 4), (9, 8210), (8211, 39993)):
        inside[a:z] = True
    assert bool((buf[~inside] == 2).all()) and bool((buf[inside] < 0.1).all())


def test_range_and_values_that_are_not_finite():
    big = torch.full((1000,), 1e30, device=DEV)
    norm = GradNorm([big]).norm()
    assert abs(float(norm) / (1e30 * 1000 ** 0.5) - 1) <= 1e-6            # squares beyond fp32's range
    small = torch.full((1000,), 1e-30, device=DEV)
    assert abs(float(GradNorm([small]).norm()) / (1e-30 * 1000 ** 0.5) - 1) <= 1e-6
    beyond = torch.full((4,), 3e38, device=DEV)
    assert float(GradNorm([beyond]).clip(1.0)) == float("inf") and bool((beyond == 0).all())
    zero = torch.zeros(5, device=DEV)
    assert float(GradNorm([zero]).clip(0.0)) == 0 and bool((zero == 0).all())
    x = torch.ones(10, device=DEV)
    GradNorm([x]).clip(0.0)
    assert bool((x == 0).all())
    for v in (float("nan"), float("inf")):
        x, y = torch.ones(9000, device=DEV), torch.ones(5, dtype=torch.bfloat16, device=DEV)
        x[8999] = v
        norm = GradNorm([x, y]).clip(1.0)
        if v != v:
            assert bool(norm.isnan()) and bool(x.isnan().all()) and bool(y.isnan().all())
        else:
            assert bool(norm.isinf()) and bool((x[:8999] == 0).all()) and bool(x[8999].isnan()) and bool((y == 0).all())
    only_empty = GradNorm([torch.empty(0, device=DEV)])
    assert float(only_empty.clip(1.0)) == 0 and float(only_empty.norm()) == 0


def test_more_than_two_to_the_31_elements():
    t = torch.full((2 ** 31 + 77,), 0.5, dtype=torch.bfloat16, device=DEV)
    t[-1] = 1024.0
    want = (0.25 * (2 ** 31 + 76) + 1024.0 ** 2) ** 0.5
    norm = GradNorm([t]).clip(0.5 * want)
    assert abs(float(norm) / want - 1) <= 2.0 ** -24
    assert float(t[-1]) == 512.0 and float(t[-2]) == 0.25 and float(t[0]) == 0.25
    assert bool((t[:-1] == 0.25).all())


def test_captured_and_replayed():
    ts = make([100, 9000, 20001], [BF, FP], 1)
    out = [torch.empty_like(t) for t in ts]
    plan, check = GradNorm(ts, out), GradNorm(ts)
    plan.clip(0.01)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = plan.clip(0.01)
    for i in range(4):
        for t in ts:
            t.normal_()
        torch.cuda.synchronize()
        graph.replay()
        again = [o.clone() for o in out]
        assert torch.equal(norm, check.norm())
        plan.clip(0.01)
        torch.cuda.synchronize()
        assert all(torch.equal(a, o) for a, o in zip(again, out))


@pytest.mark.parametrize("kind", ["object", "handle", "null"])
def test_on_a_given_stream(kind):
    ts = make([5000, 123457], [BF, FP], 2)
    plan = GradNorm(ts, [torch.empty_like(t) for t in ts])
    want = plan.clip(0.1)
    kept = [o.clone() for o in plan.out]
    for o in plan.out:
        o.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = {"object": side, "handle": side.cuda_stream, "null": 0}[kind]
    norm = plan.clip(0.1, stream=s)
    other = plan.norm(stream=s)
    torch.cuda.synchronize()
    assert torch.equal(norm, want) and torch.equal(other, want)
    assert all(torch.equal(a, o) for a, o in zip(kept, plan.out))


def other_storage(t):
    t.untyped_storage().resize_(0)


def other_data(t):
    t.data = torch.ones(300, device=DEV)


def other_set(t):
    t.set_(torch.ones(300, device=DEV))


def larger(t):
    t.resize_(1 << 22)


@pytest.mark.parametrize("change", [other_storage, other_data, other_set, larger])
def test_tensors_with_other_memory_are_refused(change):
    """Addresses are kept from the making on: a tensor whose memory is another by now is seen, and nothing is written."""
    for which, into in ((i, o) for i in range(3) for o in (False, True)):
        ts = [torch.full((n,), 2.0, device=DEV) for n in (300, 9000, 300)]
        out = [torch.full_like(t, 3.0) for t in ts] if into else None
        plan = GradNorm(ts, out)
        plan.clip(1e9)
        changed = out or ts
        change(changed[which])
        for call in (lambda: plan.norm(), lambda: plan.clip(1e-3), lambda: plan.clip(1e-3, norm=torch.ones((), device=DEV))):
            with pytest.raises(ValueError, match="memory"):
                call()
        for i, t in enumerate(changed):
            assert i == which or bool((t == 2).all())
    # tensors behind one another in one storage
    buf = torch.full((9600,), 2.0, device=DEV)
    plan = GradNorm([buf[300:], buf[:300], buf[:0]])
    norm = plan.clip(1.0)
    buf.untyped_storage().resize_(0)
    with pytest.raises(ValueError, match="memory"):
        plan.clip(1.0)
    assert abs(float(norm) - 2 * 9600 ** 0.5) <= 2e-5
    # a view that shares its storage with others and is given another: the old memory stays the object's
    a, b = torch.full((600,), 2.0, device=DEV).split(300)
    plan = GradNorm([a, b])
    b.data = torch.ones(5, device=DEV)
    assert abs(float(plan.norm()) - 2 * 600 ** 0.5) <= 1e-5


def test_a_norm_inside_the_gradients_is_refused():
    """The scaling would write it while others read it."""
    buf = torch.ones(20000, device=DEV)
    inside = GradNorm([buf[100:9000], buf[9000:19000]])
    out = torch.zeros(300, device=DEV)
    apart = GradNorm([buf[:100], buf[9000:9200]], [out[:100], out[100:]])
    for plan, refused, taken in ((inside, (100, 5000, 8999, 9000, 18999), (0, 99, 19000, 19999)),
                                 (apart, (0, 99, 9000, 9199), (100, 8999, 9200))):
        for i in refused:
            with pytest.raises(ValueError, match="norm and grads.* overlap"):
                plan.clip(0.5, norm=buf[i])
        for i in taken:
            assert plan.clip(2.0, norm=buf[i]) is not None
    with pytest.raises(ValueError, match="norm and out.0. overlap"):
        apart.clip(0.5, norm=out[99])
    assert bool((buf == 1).all())


def test_wrong_norms_and_bounds_are_refused():
    plan = GradNorm([torch.ones(4, device=DEV)])
    for norm in (1.0, torch.ones(2, device=DEV), torch.ones((), device=DEV, dtype=torch.float64), torch.ones(())):
        with pytest.raises(ValueError):
            plan.clip(1.0, norm=norm)
    for bound in (-1.0, float("nan")):
        with pytest.raises(b.MoEError):
            plan.clip(bound)
