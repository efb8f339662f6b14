"""Refusals of the serving operators' entry points, which need no GPU: host-side validation returns before
anything is enqueued, and the fake device addresses are never dereferenced."""
import pytest

from mixture_experts_layer_32_amd import binding as b

FAKE = 1 << 20


def desc(**kw):
    base = dict(T=4, H=256, F=128, E_total=8, topk=2, mode="bf16")
    base.update(kw)
    return b.Desc.make(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), "MOE_ERR_INVALID_ARG"),
    (dict(T=65), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (dict(H=384), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (dict(F=64), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (dict(E_total=513), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (dict(E_total=64, topk=33), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (dict(topk=9), "MOE_ERR_INVALID_ARG"),
    (dict(E_local=4, expert_offset=5), "MOE_ERR_INVALID_ARG"),
    (dict(mode="mxfp8"), "MOE_ERR_UNSUPPORTED_MODE"),
    (dict(mode="fp8"), "MOE_ERR_UNSUPPORTED_MODE"),
    (dict(mode=9), "MOE_ERR_UNSUPPORTED_MODE"),
])
def test_few_validation(kw, code):
    with pytest.raises(b.MoEError) as ei:
        b.query_few_sizes(desc(**kw))
    assert ei.value.code == code
    with pytest.raises(b.MoEError) as ei:
        b.moe_fwd_few(desc(**kw), FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, stream=0)
    assert ei.value.code == code


def test_few_pointers_and_workspace():
    d = desc()
    n = b.query_few_sizes(d)
    good = dict(x=FAKE, w_router=None, logits=FAKE, w_gate=FAKE, w_up=FAKE, w_down=FAKE, y=FAKE, ws=FAKE, ws_bytes=n)

    def call(**kw):
        a = {**good, **kw}
        b.moe_fwd_few(d, a["x"], a["w_router"], a["logits"], a["w_gate"], a["w_up"], a["w_down"], a["y"], a["ws"],
                      a["ws_bytes"], stream=0)

    for t in ("x", "w_gate", "w_up", "w_down", "y"):
        with pytest.raises(b.MoEError, match=f"{t} is null"):
            call(**{t: None})
        with pytest.raises(b.MoEError, match=f"{t} is not 16-byte aligned"):
            call(**{t: FAKE + 8})
    with pytest.raises(b.MoEError, match="w_router is not 16-byte aligned"):
        call(w_router=FAKE + 4)
    with pytest.raises(b.MoEError, match="logits is null"):
        call(logits=None)
    with pytest.raises(b.MoEError, match="logits is null"):
        call(logits=None, w_router=FAKE)
    with pytest.raises(b.MoEError, match="logits is not 4-byte aligned"):
        call(logits=FAKE + 2)
    with pytest.raises(b.MoEError, match="ws is not 256-byte aligned"):
        call(ws=FAKE + 16)
    with pytest.raises(b.MoEError, match="MOE_ERR_WORKSPACE_TOO_SMALL"):
        call(ws_bytes=n - 1)


@pytest.mark.parametrize("mode,elem", [("bf16", 4), ("fp32", 4)])
def test_few_workspace_holds_h_and_the_routing(mode, elem):
    T, F, E, k = 64, 768, 128, 8
    n = b.query_few_sizes(desc(T=T, F=F, E_total=E, topk=k, mode=mode))
    assert n % 256 == 0 and n >= T * k * F * elem + T * k * 4 + 8 * E


# ------------------------------------------------------------------------------------------------ 8-bit

@pytest.mark.parametrize("args,code,msg", [
    ((None, 1, 4, 64, FAKE, FAKE), "MOE_ERR_INVALID_ARG", "in is null"),
    ((FAKE, 1, 4, 64, None, FAKE), "MOE_ERR_INVALID_ARG", "q is null"),
    ((FAKE, 1, 4, 64, FAKE, None), "MOE_ERR_INVALID_ARG", "scales is null"),
    ((FAKE + 8, 1, 4, 64, FAKE, FAKE), "MOE_ERR_INVALID_ARG", "in is not 16-byte aligned"),
    ((FAKE, 1, 4, 64, FAKE + 4, FAKE), "MOE_ERR_INVALID_ARG", "q is not 16-byte aligned"),
    ((FAKE, 1, 4, 64, FAKE, FAKE + 2), "MOE_ERR_INVALID_ARG", "scales is not 4-byte aligned"),
    ((FAKE, 1, 0, 64, FAKE, FAKE), "MOE_ERR_INVALID_ARG", "positive"),
    ((FAKE, 1, 4, 0, FAKE, FAKE), "MOE_ERR_INVALID_ARG", "positive"),
    ((FAKE, 1, 4, 72, FAKE, FAKE), "MOE_ERR_UNSUPPORTED_SHAPE", "multiple of 16"),
    ((FAKE, 1, 4, 131088, FAKE, FAKE), "MOE_ERR_UNSUPPORTED_SHAPE", "131072"),
    ((FAKE, 1, 1 << 31, 16, FAKE, FAKE), "MOE_ERR_UNSUPPORTED_SHAPE", r"2\^31"),
    ((FAKE, 2, 4, 64, FAKE, FAKE), "MOE_ERR_UNSUPPORTED_MODE", "type"),
])
def test_int8_quantize_refusals(args, code, msg):
    with pytest.raises(b.MoEError, match=msg) as ei:
        b.moe_int8_quantize(*args, stream=0)
    assert ei.value.code == code


@pytest.mark.parametrize("kw,code,msg", [
    (dict(x=None), "MOE_ERR_INVALID_ARG", "x is null"),
    (dict(x=FAKE + 8), "MOE_ERR_INVALID_ARG", "x is not 16-byte aligned"),
    (dict(w=None), "MOE_ERR_INVALID_ARG", "w is null"),
    (dict(w=FAKE + 4), "MOE_ERR_INVALID_ARG", "w is not 16-byte aligned"),
    (dict(xs=None), "MOE_ERR_INVALID_ARG", "x_scales is null"),
    (dict(ws=FAKE + 1), "MOE_ERR_INVALID_ARG", "w_scales is not 4-byte aligned"),
    (dict(y=None), "MOE_ERR_INVALID_ARG", "y is null"),
    (dict(y=FAKE + 1), "MOE_ERR_INVALID_ARG", "y is not 2-byte aligned"),
    (dict(y=FAKE + 2, type=0), "MOE_ERR_INVALID_ARG", "y is not 4-byte aligned"),
    (dict(offsets=FAKE + 2), "MOE_ERR_INVALID_ARG", "offsets is not 4-byte aligned"),
    (dict(G=2), "MOE_ERR_INVALID_ARG", "offsets is null"),
    (dict(M=0), "MOE_ERR_INVALID_ARG", "positive"),
    (dict(G=0, offsets=FAKE), "MOE_ERR_INVALID_ARG", "positive"),
    (dict(K=24), "MOE_ERR_UNSUPPORTED_SHAPE", "multiple of 16"),
    (dict(K=131088), "MOE_ERR_UNSUPPORTED_SHAPE", "131072"),
    (dict(G=513, offsets=FAKE), "MOE_ERR_UNSUPPORTED_SHAPE", "512"),
    (dict(M=1 << 31), "MOE_ERR_UNSUPPORTED_SHAPE", "M must be"),
    (dict(M=(1 << 31) - 511, N=8, K=16), "MOE_ERR_UNSUPPORTED_SHAPE", "M must be"),
    (dict(N=(1 << 20) + 1), "MOE_ERR_UNSUPPORTED_SHAPE", "N <= 2"),
    (dict(M=1 << 21, N=1 << 20), "MOE_ERR_UNSUPPORTED_SHAPE", r"M\*N"),
    (dict(type=5), "MOE_ERR_UNSUPPORTED_MODE", "type"),
])
def test_int8_matmul_refusals(kw, code, msg):
    a = dict(x=FAKE, xs=FAKE, w=FAKE, ws=FAKE, M=4, N=32, K=64, G=1, offsets=None, y=FAKE, type=1)
    a.update(kw)
    with pytest.raises(b.MoEError, match=msg) as ei:
        b.moe_int8_matmul(a["x"], a["xs"], a["w"], a["ws"], a["M"], a["N"], a["K"], a["G"], a["offsets"], a["y"],
                          a["type"], stream=0)
    assert ei.value.code == code


@pytest.mark.parametrize("kw,code", [
    (dict(T=0), "MOE_ERR_INVALID_ARG"),
    (dict(H=384), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (dict(H=1 << 18), "MOE_ERR_UNSUPPORTED_SHAPE"),
    (dict(topk=9), "MOE_ERR_INVALID_ARG"),
    (dict(mode="fp32"), "MOE_ERR_UNSUPPORTED_MODE"),
    (dict(mode="mxfp8"), "MOE_ERR_UNSUPPORTED_MODE"),
])
def test_int8_layer_validation(kw, code):
    with pytest.raises(b.MoEError) as ei:
        b.query_int8_sizes(desc(**kw))
    assert ei.value.code == code


@pytest.mark.parametrize("T", [4, 300])
def test_int8_layer_pointers_and_workspace(T):
    d = desc(T=T)
    n = b.query_int8_sizes(d)
    assert n % 256 == 0 and n >= T * 2 * 128 * 4 + T * 256
    names = ("x", "w_router", "logits", "w_gate", "s_gate", "w_up", "s_up", "w_down", "s_down", "y", "ws")

    def call(ws_bytes=n, **kw):
        a = {**{k: FAKE for k in names}, "w_router": None, **kw}
        b.moe_fwd_int8(d, *(a[k] for k in names), ws_bytes, stream=0)

    for t in ("x", "w_gate", "w_up", "w_down", "y"):
        with pytest.raises(b.MoEError, match=f"{t} is null"):
            call(**{t: None})
        with pytest.raises(b.MoEError, match=f"{t} is not 16-byte aligned"):
            call(**{t: FAKE + 8})
    for t in ("s_gate", "s_up", "s_down", "logits"):
        with pytest.raises(b.MoEError, match=f"{t} is null"):
            call(**{t: None})
        with pytest.raises(b.MoEError, match=f"{t} is not 4-byte aligned"):
            call(**{t: FAKE + 2})
    with pytest.raises(b.MoEError, match="w_router is not 16-byte aligned"):
        call(w_router=FAKE + 4)
    with pytest.raises(b.MoEError, match="ws is not 256-byte aligned"):
        call(ws=FAKE + 16)
    with pytest.raises(b.MoEError, match="MOE_ERR_WORKSPACE_TOO_SMALL"):
        call(ws_bytes=n - 1)


def test_int8_layer_router_of_many_experts_and_tokens():
    d = desc(T=65, E_total=257)
    with pytest.raises(b.MoEError, match="E_total <= 256") as ei:
        b.moe_fwd_int8(d, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, stream=0)
    assert ei.value.code == "MOE_ERR_UNSUPPORTED_SHAPE"


def test_python_calls_refuse_tensors_the_library_cannot_check():
    import torch
    from mixture_experts_layer_32_amd.layer import int8_matmul, int8_quantize
    with pytest.raises(ValueError, match="dtype"):
        int8_quantize(torch.zeros(4, 16, dtype=torch.float16))
    with pytest.raises(ValueError, match="contiguous"):
        int8_quantize(torch.zeros(16, 32).t())
    with pytest.raises(ValueError, match="at least one dimension"):
        int8_quantize(torch.tensor(1.0))
    q, s = torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError, match="offsets"):
        int8_matmul(q, s, torch.zeros(2, 4, 16, dtype=torch.int8), torch.zeros(2, 4))
    with pytest.raises(ValueError, match="offsets"):
        int8_matmul(q, s, q, s, offsets=torch.zeros(2, dtype=torch.int32))
