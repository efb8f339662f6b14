"""Device-memory plumbing around the C ABI: torch allocates the caller-owned buffers.

MoELayer holds the workspace and saved buffers for one layer shape, and calls moe_fwd/moe_bwd (and
the router projection's moe_router_fwd/moe_router_bwd) through the binding. For serving, FewTokenLayer
(up to 64 tokens), Int8Layer (8-bit weights, any number of tokens), int8_quantize and int8_matmul, and
int4_quantize, int4_pack and int4_matmul. For programs that take the layer apart, sort_pairs, dispatch, combine and
combine_backward; for training steps, GradNorm. No arithmetic happens here.
"""
from __future__ import annotations

import bisect
import functools

import torch

from . import binding


def _expect(t, name, shape, dtype, device):
    """Raises ValueError unless t is a contiguous tensor of this shape and dtype on this device: the
    C ABI receives bare pointers and cannot check any of it."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")


def _on(device, stream):
    """The stream handle for a call on `device`: the given stream's, or the current one's. Raises ValueError
    unless `device` is the calling thread's current GPU, whose streams the library uses."""
    i = device.index
    # (a tensor on a GPU says that torch has initialised them: the bare call takes 0.1 us, torch.cuda.current_device 0.2)
    if device.type != "cuda" or i != torch._C._cuda_getDevice():
        raise ValueError(f"{device} is not the current GPU (torch.cuda.set_device)")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(i)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """A new output for a call on `stream`, on the device of the tensor `like`, from that stream's memory: memory of
    the current stream may still be written by work of its own."""
    if stream is None:
        # the cheapest of torch's calls for it: 1.1 to 1.3 us against 1.6 of torch.empty
        if like.shape == shape:
            return torch.empty_like(like, dtype=dtype)
        if len(shape) == 2:
            return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=like.device)
        return like.new_empty(shape, dtype=dtype)
    if isinstance(stream, int):
        # (of handle 0, the null stream's, ExternalStream would make a new stream)
        stream = torch.cuda.ExternalStream(stream, device=like.device) if stream else torch.cuda.default_stream(like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _workspace(nbytes, device):
    """Scratch memory that a layer's calls may use on any stream. torch may give memory that was freed on the current
    stream with work queued that still writes it, and a call on another stream would not be behind that work: it is
    waited for here, once. (Not while the stream is being captured, where nothing runs: such a layer's calls belong on
    the captured stream, or behind it.)"""
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    if device.type == "cuda" and not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(device).synchronize()
    return ws


def _device(device):
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


class MoELayer:
    def __init__(self, T, H, F, E_total, topk, mode="bf16", E_local=None, expert_offset=0, device="cuda",
                 recompute=False):
        """recompute=True: activation checkpointing (the backward recomputes the gate/up activations
        from x instead of reading them from the saved buffer)."""
        self.desc = binding.Desc.make(T, H, F, E_total, topk, mode, E_local, expert_offset, recompute)
        self.mode = mode
        self.dtype = torch.float32 if mode == "fp32" else torch.bfloat16
        self.device = _device(device)
        self.fwd_ws_bytes, self.bwd_ws_bytes, self.saved_bytes = binding.query_sizes(self.desc)
        self.ws = _workspace(max(self.fwd_ws_bytes, self.bwd_ws_bytes), self.device)
        self.saved = _workspace(self.saved_bytes, self.device)

    @property
    def shape(self):
        d = self.desc
        return dict(T=d.T, H=d.H, F=d.F, E=d.E_total, E_local=d.E_local, e0=d.expert_offset, k=d.topk)

    def _check(self, **tensors):
        d, el, f32 = self.desc, self.dtype, torch.float32
        spec = dict(x=((d.T, d.H), el), y=((d.T, d.H), el), dy=((d.T, d.H), el), dx=((d.T, d.H), el),
                    logits=((d.T, d.E_total), f32), dlogits=((d.T, d.E_total), f32),
                    w_gate=((d.E_local, d.F, d.H), el), w_up=((d.E_local, d.F, d.H), el),
                    w_down=((d.E_local, d.H, d.F), el), dw_gate=((d.E_local, d.F, d.H), el),
                    dw_up=((d.E_local, d.F, d.H), el), dw_down=((d.E_local, d.H, d.F), el),
                    w_router=((d.E_total, d.H), el), dw_router=((d.E_total, d.H), el))
        for name, t in tensors.items():
            shape, dtype = spec[name]
            _expect(t, name, shape, dtype, self.device)

    def forward(self, x, logits, w_gate, w_up, w_down, y=None, stream=None):
        d = self.desc
        if y is None:
            y = torch.empty(d.T, d.H, dtype=self.dtype, device=self.device)
        self._check(x=x, logits=logits, w_gate=w_gate, w_up=w_up, w_down=w_down, y=y)
        binding.moe_fwd(d, x, logits, w_gate, w_up, w_down, y, self.saved, self.ws, self.ws.numel(), stream)
        return y

    def forward_router(self, x, w_router, w_gate, w_up, w_down, y=None, logits=None, stream=None):
        """The forward from x through moe_fwd_router (router projection fused with the routing);
        returns (y, logits)."""
        d = self.desc
        if y is None:
            y = torch.empty(d.T, d.H, dtype=self.dtype, device=self.device)
        if logits is None:
            logits = torch.empty(d.T, d.E_total, dtype=torch.float32, device=self.device)
        self._check(x=x, w_router=w_router, logits=logits, w_gate=w_gate, w_up=w_up, w_down=w_down, y=y)
        binding.moe_fwd_router(d, x, w_router, logits, w_gate, w_up, w_down, y, self.saved, self.ws, self.ws.numel(),
                               stream)
        return y, logits

    def route(self, logits, stream=None):
        self._check(logits=logits)
        binding.moe_route(self.desc, logits, self.saved, self.ws, self.ws.numel(), stream)

    def backward(self, dy, x, w_gate, w_up, w_down, out=None, stream=None):
        d = self.desc
        if out is None:
            kw = dict(dtype=self.dtype, device=self.device)
            out = dict(dx=torch.empty(d.T, d.H, **kw),
                       dlogits=torch.empty(d.T, d.E_total, dtype=torch.float32, device=self.device),
                       dw_gate=torch.empty(d.E_local, d.F, d.H, **kw),
                       dw_up=torch.empty(d.E_local, d.F, d.H, **kw),
                       dw_down=torch.empty(d.E_local, d.H, d.F, **kw))
        self._check(dy=dy, x=x, w_gate=w_gate, w_up=w_up, w_down=w_down, dx=out["dx"], dlogits=out["dlogits"],
                    dw_gate=out["dw_gate"], dw_up=out["dw_up"], dw_down=out["dw_down"])
        binding.moe_bwd(d, dy, x, w_gate, w_up, w_down, self.saved, out["dx"], out["dlogits"], out["dw_gate"],
                        out["dw_up"], out["dw_down"], self.ws, self.ws.numel(), stream)
        return out

    def _router_ws(self):
        if getattr(self, "router_ws", None) is None:
            f, b = binding.query_router_sizes(self.desc)
            self.router_ws = _workspace(max(f, b, 256), self.device)
        return self.router_ws

    def router_forward(self, x, w_router, logits=None, stream=None):
        """logits = x w_router^T (fp32) through moe_router_fwd; w_router [E_total, H]."""
        d = self.desc
        if logits is None:
            logits = torch.empty(d.T, d.E_total, dtype=torch.float32, device=self.device)
        self._check(x=x, w_router=w_router, logits=logits)
        ws = self._router_ws()
        binding.moe_router_fwd(d, x, w_router, logits, ws, ws.numel(), stream)
        return logits

    def router_backward(self, x, w_router, dlogits, dx, dw_router=None, stream=None):
        """dw_router = dlogits^T x (returned), and dx += dlogits w_router in place."""
        d = self.desc
        if dw_router is None:
            dw_router = torch.empty(d.E_total, d.H, dtype=self.dtype, device=self.device)
        self._check(x=x, w_router=w_router, dlogits=dlogits, dx=dx, dw_router=dw_router)
        ws = self._router_ws()
        binding.moe_router_bwd(d, x, w_router, dlogits, dx, dw_router, ws, ws.numel(), stream)
        return dw_router

    def pairs(self):
        """Routing results in `saved` as tensors on the device, as sort_pairs, dispatch and combine name them: idx,
        weight and pair_pos [T, topk], offsets [E_local + 1], perm [T * topk] (the first offsets[-1] count). They are
        views of `saved`, which the layer's next forward or route overwrites."""
        d = self.desc
        off = binding.saved_layout(d)

        def view(name, shape, dt):
            n = 4
            for v in shape:
                n *= v
            return self.saved[off[name]:off[name] + n].view(dt).view(shape)
        tk = (d.T, d.topk)
        return dict(idx=view("idx", tk, torch.int32), weight=view("weight", tk, torch.float32),
                    offsets=view("offsets", (d.E_local + 1,), torch.int32),
                    perm=view("perm", (d.T * d.topk,), torch.int32), pair_pos=view("pair_pos", tk, torch.int32))

    def routing(self):
        """Routing results from `saved` as CPU tensors: idx, weight, counts, offsets, perm, pair_pos."""
        d = self.desc
        off = binding.saved_layout(d)
        rows = d.T * d.topk
        s = self.saved

        def view(name, n, dt):
            b = 4 * n
            return s[off[name]:off[name] + b].view(dt).cpu()
        offsets = view("offsets", d.E_local + 1, torch.int32)
        P = int(offsets[-1])
        return dict(idx=view("idx", rows, torch.int32).view(d.T, d.topk),
                    weight=view("weight", rows, torch.float32).view(d.T, d.topk),
                    counts=view("counts", d.E_local, torch.int32), offsets=offsets,
                    perm=view("perm", rows, torch.int32)[:P], pair_pos=view("pair_pos", rows, torch.int32))


class FewTokenLayer:
    """The layer's forward for 1 to 64 tokens through moe_fwd_few: holds the workspace of one shape. Calls
    of one object share it: order them, or give concurrent streams an object each, and keep an object until its
    calls have run."""

    def __init__(self, T, H, F, E_total, topk, mode="bf16", E_local=None, expert_offset=0, device="cuda"):
        self.desc = d = binding.Desc.make(T, H, F, E_total, topk, mode, E_local, expert_offset)
        self.mode = mode
        self.dtype = torch.float32 if mode == "fp32" else torch.bfloat16
        self.device = _device(device)
        self.ws = _workspace(binding.query_few_sizes(d), self.device)
        self._x, self._logits, self._wr = (d.T, d.H), (d.T, d.E_total), (d.E_total, d.H)
        self._w_in, self._w_out = (d.E_local, d.F, d.H), (d.E_local, d.H, d.F)

    def _run(self, x, w_router, logits, w_gate, w_up, w_down, y, stream):
        el, dev = self.dtype, self.device
        handle = _on(dev, stream)
        _expect(x, "x", self._x, el, dev)
        if y is None:
            y = _empty(self._x, el, x, stream)
        else:
            _expect(y, "y", self._x, el, dev)
        _expect(w_gate, "w_gate", self._w_in, el, dev)
        _expect(w_up, "w_up", self._w_in, el, dev)
        _expect(w_down, "w_down", self._w_out, el, dev)
        binding.moe_fwd_few(self.desc, x, w_router, logits, w_gate, w_up, w_down, y, self.ws, self.ws.numel(), handle)
        return y

    def forward(self, x, logits, w_gate, w_up, w_down, y=None, stream=None):
        """y of x and the router's logits [T, E_total] fp32."""
        _expect(logits, "logits", self._logits, torch.float32, self.device)
        return self._run(x, None, logits, w_gate, w_up, w_down, y, stream)

    def forward_router(self, x, w_router, w_gate, w_up, w_down, y=None, logits=None, stream=None):
        """The forward from x and w_router [E_total, H]; returns (y, logits)."""
        if logits is None:
            logits = _empty(self._logits, torch.float32, self.ws, stream)
        else:
            _expect(logits, "logits", self._logits, torch.float32, self.device)
        _expect(w_router, "w_router", self._wr, self.dtype, self.device)
        return self._run(x, w_router, logits, w_gate, w_up, w_down, y, stream), logits


_INT8_TYPES = {torch.float32: binding.TYPES["fp32"], torch.bfloat16: binding.TYPES["bf16"]}


def _int8_type(dtype):
    t = _INT8_TYPES.get(dtype)
    if t is None:
        raise ValueError(f"expected dtype torch.float32 or torch.bfloat16, got {dtype}")
    return t


def int8_quantize(x, q=None, scales=None, stream=None):
    """x [.., K] (bf16 or fp32) as signed bytes with one scale for each row of K: (q, scales), as activations
    or as the (weight, scales) pair of int8_matmul and Int8Layer."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x: expected a tensor of at least one dimension")
    t, shape, dev = _int8_type(x.dtype), x.shape, x.device
    if not x.is_contiguous():
        raise ValueError("x: expected a contiguous tensor")
    handle = _on(dev, stream)
    if q is None:
        q = _empty(shape, torch.int8, x, stream)
    else:
        _expect(q, "q", shape, torch.int8, dev)
    if scales is None:
        scales = _empty(shape[:-1], torch.float32, x, stream)
    else:
        _expect(scales, "scales", shape[:-1], torch.float32, dev)
    K = shape[-1]
    binding.moe_int8_quantize(x, t, x.numel() // K if K else 0, K, q, scales, handle)
    return q, scales


def int8_matmul(x, x_scales, w, w_scales, offsets=None, y=None, dtype=torch.bfloat16, stream=None):
    """y [M, N] of 8-bit rows x [M, K] and weights w [N, K], or w [G, N, K] with offsets [G + 1] int32: rows
    offsets[g] .. offsets[g+1]-1 are multiplied by w[g]. A y that is given sets the dtype, and its rows
    outside the groups are left as they were (a y made here holds anything there)."""
    if (not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(w, torch.Tensor)
            or w.dim() != (2 if offsets is None else 3)):
        raise ValueError("expected x [M, K] and w [N, K], or w [G, N, K] with offsets")
    dev, (M, K) = x.device, x.shape
    handle = _on(dev, stream)
    _expect(x, "x", (M, K), torch.int8, dev)
    _expect(x_scales, "x_scales", (M,), torch.float32, dev)
    if offsets is None:
        G, N = 1, w.shape[0]
        _expect(w, "w", (N, K), torch.int8, dev)
        _expect(w_scales, "w_scales", (N,), torch.float32, dev)
    else:
        G, N = w.shape[0], w.shape[1]
        _expect(w, "w", (G, N, K), torch.int8, dev)
        _expect(w_scales, "w_scales", (G, N), torch.float32, dev)
        _expect(offsets, "offsets", (G + 1,), torch.int32, dev)
    if y is None:
        t = _int8_type(dtype)
        y = _empty((M, N), dtype, x, stream)
    else:
        t = _int8_type(y.dtype)
        _expect(y, "y", (M, N), y.dtype, dev)
    binding.moe_int8_matmul(x, x_scales, w, w_scales, M, N, K, G, offsets, y, t, handle)
    return y


class Int8Layer:
    """The layer's forward with 8-bit weights through moe_fwd_int8, for any number of tokens: holds the workspace
    of one shape. Each weight is the (bytes, scales) pair of int8_quantize on the bf16 or fp32 matrix. Calls of
    one object share the workspace: order them, or give concurrent streams an object each, and keep an object until its
    calls have run."""

    def __init__(self, T, H, F, E_total, topk, E_local=None, expert_offset=0, device="cuda"):
        self.desc = d = binding.Desc.make(T, H, F, E_total, topk, "bf16", E_local, expert_offset)
        self.device = _device(device)
        self.ws = _workspace(binding.query_int8_sizes(d), self.device)
        self._x, self._logits, self._wr = (d.T, d.H), (d.T, d.E_total), (d.E_total, d.H)
        self._w_in, self._w_out = (d.E_local, d.F, d.H), (d.E_local, d.H, d.F)

    def _run(self, x, w_router, logits, w_gate, w_up, w_down, y, stream):
        dev = self.device
        handle = _on(dev, stream)
        _expect(x, "x", self._x, torch.bfloat16, dev)
        if y is None:
            y = _empty(self._x, torch.bfloat16, x, stream)
        else:
            _expect(y, "y", self._x, torch.bfloat16, dev)
        for name, (w, s), shape in (("w_gate", w_gate, self._w_in), ("w_up", w_up, self._w_in),
                                    ("w_down", w_down, self._w_out)):
            _expect(w, name, shape, torch.int8, dev)
            _expect(s, name + " scales", shape[:2], torch.float32, dev)
        binding.moe_fwd_int8(self.desc, x, w_router, logits, w_gate[0], w_gate[1], w_up[0], w_up[1], w_down[0],
                             w_down[1], y, self.ws, self.ws.numel(), handle)
        return y

    def forward(self, x, logits, w_gate, w_up, w_down, y=None, stream=None):
        """y of x and the router's logits [T, E_total] fp32; w_gate, w_up, w_down: (bytes, scales)."""
        _expect(logits, "logits", self._logits, torch.float32, self.device)
        return self._run(x, None, logits, w_gate, w_up, w_down, y, stream)

    def forward_router(self, x, w_router, w_gate, w_up, w_down, y=None, logits=None, stream=None):
        """The forward from x and w_router [E_total, H] bf16; returns (y, logits)."""
        if logits is None:
            logits = _empty(self._logits, torch.float32, self.ws, stream)
        else:
            _expect(logits, "logits", self._logits, torch.float32, self.device)
        _expect(w_router, "w_router", self._wr, torch.bfloat16, self.device)
        return self._run(x, w_router, logits, w_gate, w_up, w_down, y, stream), logits


def _matrix(t, name, types):
    """Raises ValueError unless t is a contiguous matrix of one of these dtypes; its type number otherwise."""
    if isinstance(t, torch.Tensor) and t.dim() == 2 and t.is_contiguous():
        n = types.get(t.dtype)
        if n is not None:
            return n
        raise ValueError(f"{name}: expected one of {[str(d) for d in types]}, got {t.dtype}")
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name}: expected a tensor of two dimensions")
    raise ValueError(f"{name}: expected a contiguous tensor")


_DISPATCH_TYPES = {**_INT8_TYPES, torch.int8: binding.TYPES["int8"]}


@functools.lru_cache(maxsize=256)
def _sort_bytes(pairs, E_local, expert_offset):
    if not -2 ** 31 <= E_local < 2 ** 31 or not -2 ** 31 <= expert_offset < 2 ** 31:
        raise ValueError("E_local and expert_offset: expected 32-bit numbers")
    return binding.query_sort_sizes(pairs, E_local)


def sort_pairs(idx, E_local, expert_offset=0, stream=None):
    """The (token, slot) pairs sorted by expert: idx [T, topk] int32 names each pair's expert (of any router; -1 or
    another rank's: no position). Returns offsets [E_local + 1], perm [T * topk] and pair_pos [T, topk], int32: the
    first position of each expert's pairs, the pair at each position (-1 behind the last), and each pair's position
    (-1: none)."""
    if not isinstance(idx, torch.Tensor) or idx.dim() != 2:
        raise ValueError("idx: expected a tensor of two dimensions")
    shape, dev, n = idx.shape, idx.device, idx.numel()
    handle = _on(dev, stream)
    _expect(idx, "idx", shape, torch.int32, dev)
    ws_bytes = _sort_bytes(n, E_local, expert_offset)
    # one allocation and three views: 1 us less than three
    offsets, perm, pair_pos = _empty((E_local + 1 + 2 * n,), torch.int32, idx, stream).split_with_sizes((E_local + 1, n, n))
    ws = _empty((ws_bytes,), torch.uint8, idx, stream) if ws_bytes else None
    binding.moe_sort_pairs(idx, n, E_local, expert_offset, offsets, perm, pair_pos, ws, ws_bytes, handle)
    return offsets, perm, pair_pos.view(shape)


def dispatch(x, pair_pos, rows=None, stream=None):
    """rows[pair_pos[t, j]] = x[t] for x [T, H] (bf16, fp32 or int8) and pair_pos [T, topk] int32. rows [n, H] is
    [T * topk, H] unless it is given; rows that no pair stands at are left as they were (rows made here hold anything
    there). The gradient with respect to x is combine(drows, pair_pos)."""
    t = _matrix(x, "x", _DISPATCH_TYPES)
    dev, (T, H) = x.device, x.shape
    handle = _on(dev, stream)
    k = pair_pos.shape[-1] if isinstance(pair_pos, torch.Tensor) and pair_pos.dim() == 2 else 0
    _expect(pair_pos, "pair_pos", (T, k), torch.int32, dev)
    if rows is None:
        rows = _empty((T * k, H), x.dtype, x, stream)
    else:
        _matrix(rows, "rows", _DISPATCH_TYPES)
        _expect(rows, "rows", (rows.shape[0], H), x.dtype, dev)
    binding.moe_dispatch(x, t, T, k, H, pair_pos, rows, rows.shape[0], handle)
    return rows


def combine(rows, pair_pos, weight=None, y=None, dtype=None, stream=None):
    """y[t] = sum over the slots j with a position of weight[t, j] rows[pair_pos[t, j]] (weight None: 1), in fp32 and
    rounded once: rows [n, H] (bf16 or fp32), pair_pos [T, topk] int32, weight [T, topk] fp32, y [T, H] of dtype
    (rows' own if None)."""
    rt = _matrix(rows, "rows", _INT8_TYPES)
    dev, (n, H) = rows.device, rows.shape
    handle = _on(dev, stream)
    shape = pair_pos.shape if isinstance(pair_pos, torch.Tensor) else ()
    if len(shape) != 2:
        raise ValueError("pair_pos: expected a tensor of two dimensions")
    _expect(pair_pos, "pair_pos", shape, torch.int32, dev)
    if weight is not None:
        _expect(weight, "weight", shape, torch.float32, dev)
    T, k = shape
    if y is None:
        if dtype is None or dtype is rows.dtype:
            dtype, t = rows.dtype, rt
        else:
            t = _int8_type(dtype)
        y = _empty((T, H), dtype, rows, stream)
    else:
        t = _matrix(y, "y", _INT8_TYPES)
        _expect(y, "y", (T, H), y.dtype if dtype is None else dtype, dev)
    binding.moe_combine(rows, rt, n, pair_pos, weight, T, k, H, y, t, handle)
    return y


def combine_backward(dy, rows, weight, pair_pos, idx=None, E_total=None, drows=None, stream=None):
    """The gradients of combine(rows, pair_pos, weight) for dy [T, H]: (drows, dweight), and with the pairs' experts idx
    [T, topk] int32 and E_total also dlogits [T, E_total] fp32, for weights that are a softmax over the chosen experts'
    logits. drows [n, H] is of rows' type; its rows that no pair stands at are left as they were."""
    rt, t = _matrix(rows, "rows", _INT8_TYPES), _matrix(dy, "dy", _INT8_TYPES)
    dev, (n, H), T = rows.device, rows.shape, dy.shape[0]
    handle = _on(dev, stream)
    k = pair_pos.shape[-1] if isinstance(pair_pos, torch.Tensor) and pair_pos.dim() == 2 else 0
    _expect(pair_pos, "pair_pos", (T, k), torch.int32, dev)
    _expect(dy, "dy", (T, H), dy.dtype, dev)
    _expect(weight, "weight", (T, k), torch.float32, dev)
    if (idx is None) != (E_total is None):
        raise ValueError("expected both idx and E_total, or neither")
    if idx is not None:
        _expect(idx, "idx", (T, k), torch.int32, dev)
        if not 0 < E_total < 2 ** 31:
            raise ValueError(f"E_total: expected a positive 32-bit number, got {E_total}")
    if drows is None:
        drows = _empty((n, H), rows.dtype, rows, stream)
    else:
        _expect(drows, "drows", (n, H), rows.dtype, dev)
    dweight = _empty((T, k), torch.float32, weight, stream)
    dlogits = _empty((T, E_total), torch.float32, rows, stream) if idx is not None else None
    binding.moe_combine_bwd(dy, t, rows, rt, n, pair_pos, weight, idx, T, k, H, E_total or 0, drows, dweight, dlogits,
                            handle)
    return (drows, dweight) if idx is None else (drows, dweight, dlogits)


def _int4_out(shape, group, like, stream):
    """New tiles and scales of a weight [.., N, K] in 4 bits."""
    *lead, N, K = shape
    if group not in (32, 64, 128):
        raise ValueError(f"group: expected 32, 64 or 128, got {group}")
    rows, cols = -(-N // 64), -(-K // 128)
    return (_empty((*lead, rows, 4096 * cols + 16), torch.uint8, like, stream),
            _empty((*lead, rows, cols, 64, 128 // group), torch.bfloat16, like, stream))


def _int4_shape(w, name):
    if not isinstance(w, torch.Tensor) or w.dim() not in (2, 3):
        raise ValueError(f"{name}: expected [N, K] or [G, N, K]")
    if not w.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return 1 if w.dim() == 2 else w.shape[0], w.shape[-2], w.shape[-1]


def int4_quantize(w, group=128, stream=None):
    """A weight w [N, K] or [G, N, K] (bf16 or fp32) in 4 bits with a bf16 scale for each `group` (32, 64 or 128) inputs:
    the (tiles, scales) pair that int4_matmul takes."""
    G, N, K = _int4_shape(w, "w")
    t, handle = _int8_type(w.dtype), _on(w.device, stream)
    q, s = _int4_out(w.shape, group, w, stream)
    binding.moe_int4_quantize(w, t, G, N, K, group, q, s, handle)
    return q, s


def int4_pack(values, scales, stream=None):
    """The (tiles, scales) pair of a weight that is quantised already: values [N, K] or [G, N, K] int8, whole numbers of
    -8..7, and scales [.., N, K / group] bf16."""
    G, N, K = _int4_shape(values, "values")
    dev = values.device
    handle = _on(dev, stream)
    _expect(values, "values", values.shape, torch.int8, dev)
    n = scales.shape[-1] if isinstance(scales, torch.Tensor) and scales.dim() else 0
    _expect(scales, "scales", (*values.shape[:-1], n), torch.bfloat16, dev)
    group = K // n if n and K % n == 0 else 0
    q, s = _int4_out(values.shape, group, values, stream)
    binding.moe_int4_pack(values, scales, G, N, K, group, q, s, handle)
    return q, s


def int4_matmul(x, q, scales, offsets=None, N=None, y=None, dtype=torch.bfloat16, stream=None):
    """y [M, N] of bf16 rows x [M, K] and a weight in 4 bits, (q, scales) of int4_quantize or int4_pack on [N, K], or
    on [G, N, K] with offsets [G + 1] int32: rows offsets[g] .. offsets[g+1]-1 are multiplied by weight g. N is
    needed where it is no multiple of 64 (and y is not given). The weight's K is checked here to whole 128 inputs; y is
    NaN where x has another K than the weight within them. A y that is given sets the dtype, and its rows outside
    the groups are left as they were (a y made here holds anything there)."""
    if (not isinstance(x, torch.Tensor) or x.dim() != 2 or not isinstance(q, torch.Tensor)
            or q.dim() != (2 if offsets is None else 3) or not isinstance(scales, torch.Tensor)
            or scales.dim() != q.dim() + 2):
        raise ValueError("expected x [M, K] and (q, scales) of a weight [N, K], or of [G, N, K] with offsets")
    dev, (M, K) = x.device, x.shape
    handle = _on(dev, stream)
    _expect(x, "x", (M, K), torch.bfloat16, dev)
    cols, ng = -(-K // 128), scales.shape[-1]
    if ng not in (1, 2, 4):
        raise ValueError(f"scales: expected 1, 2 or 4 for each 128 inputs, got {ng}")
    if offsets is None:
        G, rows = 1, q.shape[0]
        _expect(q, "q", (rows, 4096 * cols + 16), torch.uint8, dev)
        _expect(scales, "scales", (rows, cols, 64, ng), torch.bfloat16, dev)
    else:
        G, rows, _ = q.shape
        _expect(q, "q", (G, rows, 4096 * cols + 16), torch.uint8, dev)
        _expect(scales, "scales", (G, rows, cols, 64, ng), torch.bfloat16, dev)
        _expect(offsets, "offsets", (G + 1,), torch.int32, dev)
    if N is None:
        N = y.shape[-1] if isinstance(y, torch.Tensor) and y.dim() else 64 * rows
    if -(-N // 64) != rows:
        raise ValueError(f"N: {N} channels are not {rows} times 64, or up to 63 less")
    if y is None:
        t = _int8_type(dtype)
        y = _empty((M, N), dtype, x, stream)
    else:
        t = _int8_type(y.dtype)
        _expect(y, "y", (M, N), y.dtype, dev)
    binding.moe_int4_matmul(x, q, scales, M, N, K, 128 // ng, G, offsets, y, t, handle)
    return y


class GradNorm:
    """The norm over many gradients together, and their scaling so that it stays within a bound: holds the list of
    tensors, their addresses and the workspace, for gradients that stay in place from step to step. Gradients that are new
    tensors at each step need a new object each (1.5 to 3 us of host time a tensor), or buffers that they are copied to. A
    tensor whose storage was resized, or which has been given another one, is refused at the next call (of tensors that
    share a storage, the first is looked at). Calls of one object share the workspace: order them, or give concurrent
    streams an object each, and keep an object until its calls, and the replays of a graph that holds one, have run."""

    def __init__(self, grads, out=None):
        """grads: contiguous bf16 and fp32 tensors on the current GPU, which may not overlap. out: where the scaled
        gradients go (the same sizes, either type), or None for in place."""
        self.grads = list(grads)
        self.out = None if out is None else list(out)
        if not self.grads:
            raise ValueError("grads: expected at least one tensor")
        if self.out is not None and len(self.out) != len(self.grads):
            raise ValueError(f"out: expected {len(self.grads)} tensors, got {len(self.out)}")
        self.device = self.grads[0].device if isinstance(self.grads[0], torch.Tensor) else torch.device("cpu")
        self._in = self._table(self.grads, "grads")
        self._out = None if self.out is None else self._table(self.out, "out")
        spans = []
        for i, g in enumerate(self.grads):
            o = g if self.out is None else self.out[i]
            if o.numel() != g.numel():
                raise ValueError(f"out[{i}]: expected {g.numel()} elements, got {o.numel()}")
            spans.append((g.data_ptr(), g.numel() * g.element_size(), f"grads[{i}]"))
            if o.data_ptr() != g.data_ptr() or o.dtype != g.dtype:
                spans.append((o.data_ptr(), o.numel() * o.element_size(), f"out[{i}]"))
        self._spans = spans = sorted(s for s in spans if s[1])
        for (a, n, name), (b, _, other) in zip(spans, spans[1:]):
            if b < a + n:
                raise ValueError(f"{name} and {other} overlap")
        # The storages that the addresses lie in are kept, so that they stay memory of these tensors, and one tensor of
        # each is asked for its address at every call: a storage that is resized has another.
        self._storages, self._watched = {}, []
        for t in self.grads + (self.out or []):
            s = t.untyped_storage()
            if t.numel() and s._cdata not in self._storages:
                self._storages[s._cdata] = s
                self._watched.append((t.data_ptr, t.data_ptr()))
        self.ws = _workspace(max(256, binding.query_norm_sizes(self._in, len(self.grads))), self.device)

    def _in_place(self):
        for address, was in self._watched:
            if address() != was:
                raise ValueError("a tensor's memory is another than when the object was made: make a new one")

    def _table(self, tensors, name):
        table = (binding.Tensor * len(tensors))()
        for i, t in enumerate(tensors):
            if not isinstance(t, torch.Tensor):
                raise ValueError(f"{name}[{i}]: expected a torch.Tensor, got {type(t).__name__}")
            _expect(t, f"{name}[{i}]", t.shape, t.dtype, self.device)
            table[i] = binding.Tensor(t.data_ptr(), t.numel(), _int8_type(t.dtype))
        return table

    def norm(self, stream=None):
        """The norm, an fp32 tensor without dimensions on the device."""
        handle = _on(self.device, stream)
        self._in_place()
        norm = _empty((), torch.float32, self.ws, stream)
        binding.moe_grad_norm(self._in, len(self.grads), norm, self.ws, self.ws.numel(), handle)
        return norm

    def clip(self, max_norm, norm=None, stream=None):
        """Scales the gradients by min(1, max_norm / (norm + 1e-6)) and returns the norm: their own, or the one given (an
        fp32 tensor of one element outside of the gradients, such as a norm over all ranks')."""
        handle = _on(self.device, stream)
        self._in_place()
        n = len(self.grads)
        if norm is None:
            norm = _empty((), torch.float32, self.ws, stream)
            binding.moe_clip_grad_norm(self._in, self._out, n, max_norm, norm, self.ws, self.ws.numel(), handle)
            return norm
        if not isinstance(norm, torch.Tensor) or norm.numel() != 1:
            raise ValueError("norm: expected a tensor of one element")
        _expect(norm, "norm", norm.shape, torch.float32, self.device)
        # (the scaling reads it while it writes the gradients)
        i = bisect.bisect_right(self._spans, (norm.data_ptr() + 3,)) - 1
        if i >= 0 and norm.data_ptr() < self._spans[i][0] + self._spans[i][1]:
            raise ValueError(f"norm and {self._spans[i][2]} overlap")
        binding.moe_grad_clip(self._in, self._out, n, norm, max_norm, handle)
        return norm
