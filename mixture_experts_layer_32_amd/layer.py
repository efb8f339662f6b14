"""Device-memory plumbing around the C ABI: torch allocates the caller-owned buffers.

MoELayer holds the workspace and saved buffers for one layer shape, and calls moe_fwd/moe_bwd (and
the router projection's moe_router_fwd/moe_router_bwd) through the binding. For serving, FewTokenLayer
(up to 64 tokens), Int8Layer (8-bit weights, any number of tokens), int8_quantize and int8_matmul. No
arithmetic happens here.
"""
from __future__ import annotations

import torch

from . import binding


def _expect(t, name, shape, dtype, device):
    """Raises ValueError unless t is a contiguous tensor of this shape and dtype on this device: the
    C ABI receives bare pointers and cannot check any of it."""
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous():
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
    if device.type != "cuda" or i != torch.cuda.current_device():
        raise ValueError(f"{device} is not the current GPU (torch.cuda.set_device)")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(i)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(shape, dtype, like, stream):
    """A new output for a call on `stream`, on the device of the tensor `like`, from that stream's memory: memory of
    the current stream may still be written by work of its own."""
    if stream is None:
        # the cheapest of torch's calls for it: 0.9 us against 1.4 of torch.empty
        return torch.empty_like(like, dtype=dtype) if like.shape == shape else like.new_empty(shape, dtype=dtype)
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
