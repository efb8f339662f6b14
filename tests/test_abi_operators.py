"""Refusals of the entry points for sorted pairs, 4-bit weights and gradient norms, which need no GPU: host-side
validation returns before anything is enqueued, and the fake device addresses are never dereferenced."""
import ctypes

import pytest
import torch

from mixture_experts_layer_32_amd import binding as b
from mixture_experts_layer_32_amd import layer

FAKE = 1 << 20
SHAPE, ARG, MODE = "MOE_ERR_UNSUPPORTED_SHAPE", "MOE_ERR_INVALID_ARG", "MOE_ERR_UNSUPPORTED_MODE"
WS = "MOE_ERR_WORKSPACE_TOO_SMALL"


def refused(code, call, match=None):
    with pytest.raises(b.MoEError, match=match) as ei:
        call()
    assert ei.value.code == code


def test_every_declared_function_has_its_argument_types():
    L = b.lib()
    for n in b.header_functions():
        f = getattr(L, n)
        assert f.argtypes is not None or n in ("moe_version", "moe_profile_disable", "moe_profile_collect"), n


def sort(pairs=5000, E_local=8, expert_offset=0, **kw):
    a = dict(idx=FAKE, offsets=FAKE, perm=FAKE, pair_pos=FAKE, ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    b.moe_sort_pairs(a["idx"], pairs, E_local, expert_offset, a["offsets"], a["perm"], a["pair_pos"], a["ws"],
                     a["ws_bytes"], stream=0)


@pytest.mark.parametrize("pairs,E_local,code", [(-1, 8, ARG), (-3, 8, ARG), (8, 0, ARG), (8, 513, SHAPE),
                                                (1 << 31, 8, SHAPE)])
def test_sort_sizes(pairs, E_local, code):
    refused(code, lambda: b.query_sort_sizes(pairs, E_local))
    refused(code, lambda: sort(pairs, E_local))


def test_sort_arguments():
    refused(ARG, lambda: sort(expert_offset=-1))
    for t in ("idx", "offsets", "perm", "pair_pos"):
        refused(ARG, lambda: sort(**{t: None}), f"{t} is null")
        refused(ARG, lambda: sort(**{t: FAKE + 2}), f"{t} is not 4-byte aligned")
    n = b.query_sort_sizes(5000, 8)
    assert n > 0 and n % 256 == 0
    refused(WS, lambda: sort(ws_bytes=n - 1))
    refused(ARG, lambda: sort(ws=None), "ws is null")
    refused(ARG, lambda: sort(ws=FAKE + 128), "ws is not 256-byte aligned")
    assert b.query_sort_sizes(1, 512) == 0


def dispatch(type=1, T=4, topk=2, H=16, nrows=8, **kw):
    a = dict(x=FAKE, pair_pos=FAKE, rows=FAKE)
    a.update(kw)
    b.moe_dispatch(a["x"], type, T, topk, H, a["pair_pos"], a["rows"], nrows, stream=0)


def combine(rows_type=1, type=1, T=4, topk=2, H=16, nrows=8, **kw):
    a = dict(rows=FAKE, pair_pos=FAKE, weight=FAKE, y=FAKE)
    a.update(kw)
    b.moe_combine(a["rows"], rows_type, nrows, a["pair_pos"], a["weight"], T, topk, H, a["y"], type, stream=0)


def combine_bwd(rows_type=1, type=1, T=4, topk=2, H=16, nrows=8, E_total=8, **kw):
    a = dict(dy=FAKE, rows=FAKE, pair_pos=FAKE, weight=FAKE, idx=FAKE, drows=FAKE, dweight=FAKE, dlogits=FAKE)
    a.update(kw)
    b.moe_combine_bwd(a["dy"], type, a["rows"], rows_type, nrows, a["pair_pos"], a["weight"], a["idx"], T, topk, H,
                      E_total, a["drows"], a["dweight"], a["dlogits"], stream=0)


@pytest.mark.parametrize("call", [dispatch, combine, combine_bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), ARG), (dict(topk=0), ARG), (dict(H=0), ARG), (dict(nrows=-1), ARG), (dict(topk=33), SHAPE),
    (dict(T=1 << 28, topk=8), SHAPE), (dict(T=1 << 62), SHAPE), (dict(H=1 << 40), SHAPE), (dict(H=1 << 62), SHAPE),
    (dict(H=1 << 30, nrows=1 << 10), SHAPE), (dict(type=3), MODE), (dict(type=-1), MODE),
])
def test_pairs_sizes(call, kw, code):
    refused(code, lambda: call(**kw))


def test_pairs_arguments():
    for t in ("x", "rows"):
        refused(ARG, lambda: dispatch(**{t: None}), f"{t} is null")
        refused(ARG, lambda: dispatch(**{t: FAKE + 1}), f"{t} is not 2-byte aligned")
        refused(ARG, lambda: dispatch(type=0, **{t: FAKE + 2}), f"{t} is not 4-byte aligned")
    refused(ARG, lambda: dispatch(pair_pos=FAKE + 2), "pair_pos is not 4-byte aligned")
    for t in ("rows", "pair_pos", "y"):
        refused(ARG, lambda: combine(**{t: None}), f"{t} is null")
    refused(ARG, lambda: combine(weight=FAKE + 2), "weight is not 4-byte aligned")
    refused(ARG, lambda: combine(rows_type=0, rows=FAKE + 2), "rows is not 4-byte aligned")
    refused(MODE, lambda: combine(rows_type=2))
    refused(MODE, lambda: combine(type=2))
    for t in ("dy", "rows", "drows", "pair_pos", "weight", "dweight", "idx"):
        refused(ARG, lambda: combine_bwd(**{t: None}), f"{t} is null")
    refused(ARG, lambda: combine_bwd(E_total=0), "E_total")
    refused(SHAPE, lambda: combine_bwd(E_total=513), "E_total")
    refused(MODE, lambda: combine_bwd(rows_type=2))


def test_pairs_sizes_up_to_the_limit():
    """T*H and nrows*H just below 2^40 (3 divides 2^40 - 1), in calls that have nothing to do."""
    H = (2 ** 40 - 1) // 3
    dispatch(T=3, H=H, nrows=0, rows=None)
    combine(T=0, H=H, nrows=3)
    combine_bwd(T=0, H=H, nrows=3)
    for call in (lambda h: dispatch(T=3, H=h, nrows=0, rows=None), lambda h: combine(T=0, H=h, nrows=3),
                 lambda h: combine_bwd(T=0, H=h, nrows=3)):
        refused(SHAPE, lambda: call(H + 1), "2\\^40")


def test_without_tokens_or_rows_there_is_nothing_to_do():
    dispatch(T=0, x=None, pair_pos=None)
    dispatch(nrows=0, rows=None)
    combine(T=0, y=None, pair_pos=None, weight=None)
    combine_bwd(T=0, dy=None, pair_pos=None, weight=None, idx=None, dweight=None, dlogits=None)


def matmul(M=4, N=16, K=128, group=32, G=1, type=1, **kw):
    a = dict(x=FAKE, q=FAKE, scales=FAKE, offsets=None if G == 1 else FAKE, y=FAKE)
    a.update(kw)
    b.moe_int4_matmul(a["x"], a["q"], a["scales"], M, N, K, group, G, a["offsets"], a["y"], type, stream=0)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), ARG), (dict(K=0), ARG), (dict(G=0), ARG), (dict(group=16), SHAPE), (dict(group=0), SHAPE),
    (dict(group=-32), SHAPE), (dict(K=48), SHAPE), (dict(K=96, group=64), SHAPE), (dict(K=131072 + 32), SHAPE),
    (dict(N=(1 << 20) + 1), SHAPE), (dict(G=513), SHAPE), (dict(G=512, N=1 << 20, K=2048), SHAPE),
])
def test_int4_sizes(kw, code):
    a = {**dict(G=1, N=16, K=128, group=32), **kw}
    refused(code, lambda: b.query_int4_sizes(a["G"], a["N"], a["K"], a["group"]))
    refused(code, lambda: b.moe_int4_quantize(FAKE, 1, a["G"], a["N"], a["K"], a["group"], FAKE, FAKE, stream=0))
    refused(code, lambda: b.moe_int4_pack(FAKE, FAKE, a["G"], a["N"], a["K"], a["group"], FAKE, FAKE, stream=0))
    refused(code, lambda: matmul(**kw))


def test_int4_arguments():
    assert b.query_int4_sizes(3, 65, 160, 32) == (3 * 2 * (2 * 4096 + 16), 3 * 2 * 2 * 64 * 4 * 2)
    refused(ARG, lambda: matmul(M=-1))
    matmul(M=0, x=None, y=None)                    # no rows: nothing to do
    refused(SHAPE, lambda: matmul(M=1 << 31))
    refused(SHAPE, lambda: matmul(M=1 << 30, N=1 << 10))
    refused(MODE, lambda: matmul(type=2))
    refused(ARG, lambda: matmul(G=2, offsets=None), "offsets is null")
    for t, a in (("x", 16), ("q", 16), ("scales", 16), ("y", 2)):
        refused(ARG, lambda: matmul(**{t: None}), f"{t} is null")
        refused(ARG, lambda: matmul(**{t: FAKE + a // 2}), f"{t} is not {a}-byte aligned")
    refused(ARG, lambda: matmul(type=0, y=FAKE + 2), "y is not 4-byte aligned")
    refused(MODE, lambda: b.moe_int4_quantize(FAKE, 2, 1, 16, 128, 32, FAKE, FAKE, stream=0))
    refused(ARG, lambda: b.moe_int4_quantize(None, 1, 1, 16, 128, 32, FAKE, FAKE, stream=0), "in is null")
    refused(ARG, lambda: b.moe_int4_pack(FAKE, None, 1, 16, 128, 32, FAKE, FAKE, stream=0), "in_scales is null")


def table(*entries):
    return (b.Tensor * len(entries))(*[b.Tensor(*e) for e in entries])


@pytest.mark.parametrize("entry,code", [
    ((FAKE, -1, 1), ARG), ((None, 5, 1), ARG), ((FAKE + 2, 5, 0), ARG), ((FAKE + 1, 5, 1), ARG), ((FAKE, 5, 2), MODE),
    ((FAKE, 1 << 40, 1), SHAPE), ((FAKE, (1 << 40) - 6, 1), SHAPE),
])
def test_norm_tensors(entry, code):
    t = table((FAKE, 6, 0), entry)
    refused(code, lambda: b.query_norm_sizes(t, 2), r"tensors")
    refused(code, lambda: b.moe_grad_norm(t, 2, FAKE, FAKE, 1 << 40, stream=0))
    refused(code, lambda: b.moe_grad_clip(t, None, 2, FAKE, 1.0, stream=0))
    refused(code, lambda: b.moe_clip_grad_norm(t, None, 2, 1.0, FAKE, FAKE, 1 << 40, stream=0))


def test_norm_arguments():
    t = table((FAKE, 6, 0), (None, 0, 1), (FAKE + 64, 70000, 1))
    n = b.query_norm_sizes(t, 3)
    assert n >= 8 * 10 and n % 256 == 0
    assert b.query_norm_sizes(None, 0) == 0
    refused(ARG, lambda: b.query_norm_sizes(None, 1), "tensors is null")
    refused(ARG, lambda: b.query_norm_sizes(t, -1), "count")
    for f in (lambda **kw: b.moe_grad_norm(t, 3, kw.get("norm", FAKE), kw.get("ws", FAKE), kw.get("n", n), stream=0),
              lambda **kw: b.moe_clip_grad_norm(t, None, 3, 1.0, kw.get("norm", FAKE), kw.get("ws", FAKE),
                                                kw.get("n", n), stream=0)):
        refused(ARG, lambda: f(norm=None), "norm is null")
        refused(ARG, lambda: f(ws=None), "ws is null")
        refused(ARG, lambda: f(ws=FAKE + 64), "ws is not 256-byte aligned")
        refused(WS, lambda: f(n=n - 1))
    for max_norm in (-1.0, float("nan")):
        refused(ARG, lambda: b.moe_grad_clip(t, None, 3, FAKE, max_norm, stream=0), "max_norm")
        refused(ARG, lambda: b.moe_clip_grad_norm(t, None, 3, max_norm, FAKE, FAKE, n, stream=0), "max_norm")
    refused(ARG, lambda: b.moe_grad_clip(t, None, 3, None, 1.0, stream=0), "norm is null")
    other = table((FAKE, 6, 0), (None, 0, 1), (FAKE + 64, 70001, 1))
    refused(ARG, lambda: b.moe_grad_clip(t, other, 3, FAKE, 1.0, stream=0), "another size")
    other = table((FAKE, 6, 1), (None, 0, 1), (FAKE + 64, 70000, 1))
    refused(ARG, lambda: b.moe_grad_clip(t, other, 3, FAKE, 1.0, stream=0), "in another type")
    refused(MODE, lambda: b.moe_grad_clip(t, table((FAKE, 6, 5), (None, 0, 1), (FAKE, 70000, 1)), 3, FAKE, 1.0, stream=0))


def test_tensors_off_the_gpu_are_refused():
    i = torch.zeros((4, 2), dtype=torch.int32)
    x = torch.zeros((4, 16), dtype=torch.bfloat16)
    calls = [lambda: layer.sort_pairs(i, 8), lambda: layer.dispatch(x, i), lambda: layer.combine(x, i),
             lambda: layer.combine_backward(x, x, torch.zeros(4, 2), i), lambda: layer.int4_quantize(x),
             lambda: layer.int4_pack(torch.zeros((4, 32), dtype=torch.int8), torch.zeros((4, 1), dtype=torch.bfloat16)),
             lambda: layer.int4_matmul(x, torch.zeros((1, 4112), dtype=torch.uint8),
                                       torch.zeros((1, 1, 64, 1), dtype=torch.bfloat16)),
             lambda: layer.GradNorm([x]).norm()]
    for c in calls:
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            c()


def test_grad_norm_refuses_what_it_cannot_hold():
    x = torch.zeros(64)
    with pytest.raises(ValueError, match="at least one"):
        layer.GradNorm([])
    with pytest.raises(ValueError, match="contiguous"):
        layer.GradNorm([x[::2]])
    with pytest.raises(ValueError, match="float64"):
        layer.GradNorm([x.double()])
    with pytest.raises(ValueError, match="expected a torch.Tensor"):
        layer.GradNorm([x, 3])
    with pytest.raises(ValueError, match="overlap"):
        layer.GradNorm([x[:33], x[32:]])
    with pytest.raises(ValueError, match="overlap"):
        layer.GradNorm([x, x])
    with pytest.raises(ValueError, match="overlap"):
        layer.GradNorm([x[:32], x[32:]], [x[1:33], torch.zeros(32)])
    with pytest.raises(ValueError, match="expected 2 tensors"):
        layer.GradNorm([x[:32], x[32:]], [x[:32]])
    with pytest.raises(ValueError, match="expected 64 elements"):
        layer.GradNorm([x], [x[:32]])
    layer.GradNorm([x[:32], x[32:], x[:0]], [x[:32], torch.zeros(32, dtype=torch.bfloat16), x[:0]])
