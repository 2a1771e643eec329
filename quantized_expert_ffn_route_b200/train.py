"""Training side of the binding: the calls of include/moe_train.h, and one
layer's training step made of them.

The functions named moe_* forward to the C calls of the same name.  Device
buffers are torch CUDA tensors (or raw integer pointers, taken as they are):
a tensor has to be contiguous, of the call's type, large enough and on the
device of the call's other tensors, else ValueError; the call runs on that
device, on `stream` or the device's current stream.
"""
from __future__ import annotations

import ctypes as C

MOE_Q8 = 2          # activation given as an 8-bit checkpoint (codes, scales)

_P, _I, _F, _Z = C.c_void_p, C.c_int, C.c_float, C.c_size_t
SIGNATURES = {
    "moe_act_pack8": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_act_unpack8": (_I, [_P, _P, _I, _I, _P, _I, _P]),
    "moe_balance_ws_size": (_Z, [_I, _I]),
    "moe_balance_loss": (_I, [_P, _P, _P, _I, _I, _I, _F, _F, _P, _P, _P, _Z, _P]),
    "moe_route_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _F, _F, _P, _I, _P]),
    "moe_expert_ffn_backward_ws_size": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "moe_expert_ffn_backward": (_I, [_I, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _I,
                                     _P, _I, _P, _Z, _P]),
    "moe_router_backward_ws_size": (_Z, [_I, _I, _I, _I, _I, _I]),
    "moe_router_backward": (_I, [_P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _P, _I, _P, _P, _P, _Z, _P]),
}


class _Call:
    """Checks one call's tensors and runs it on their device."""

    def __init__(self, name):
        self.name, self.device = name, None

    def ptr(self, t, what, dtypes, count):
        """Pointer of a buffer of at least `count` values; None and integers pass."""
        if t is None or isinstance(t, int):
            return t
        import torch
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{self.name}: {what} must be a CUDA tensor, an address or None (got {type(t).__name__})")
        if not t.is_cuda:
            raise ValueError(f"{self.name}: {what} must be a CUDA tensor (got {t.device})")
        if t.dtype not in dtypes:
            raise ValueError(f"{self.name}: {what} has type {t.dtype}, expected {' or '.join(map(str, dtypes))}")
        if not t.is_contiguous():
            raise ValueError(f"{self.name}: {what} must be contiguous")
        if t.numel() < count:
            raise ValueError(f"{self.name}: {what} holds {t.numel()} values, needs {count}")
        if self.device is None:
            self.device = t.device
        elif self.device != t.device:
            raise ValueError(f"{self.name}: {what} is on {t.device}, other buffers on {self.device}")
        return t.data_ptr()

    def run(self, stream, *args):
        from . import _check, _stream, lib
        import torch
        fn = getattr(lib(), self.name)
        if self.device is None or self.device.index == torch.cuda.current_device():
            return _check(fn(*args, _stream(stream)))
        with torch.cuda.device(self.device):
            return _check(fn(*args, _stream(stream)))


_TYPES = None


def _types(code):
    """torch types of a dtype code (an unknown code passes: the C call refuses it)."""
    global _TYPES
    if _TYPES is None:
        import torch
        _TYPES = {0: (torch.float32,), 1: (torch.bfloat16,), MOE_Q8: (torch.int8,), "i32": (torch.int32,),
                  "i64": (torch.int64,), "u8": (torch.uint8,), "mask": (torch.uint8, torch.bool),
                  None: (torch.float32, torch.bfloat16, torch.int8)}
    return _TYPES.get(code, _TYPES[None])


def moe_act_pack8(x, x_dtype, T, H, codes, scales, stream=None):
    c = _Call("moe_act_pack8")
    return c.run(stream, c.ptr(x, "x", _types(x_dtype), T * H), x_dtype, T, H,
                 c.ptr(codes, "codes", _types(MOE_Q8), T * H), c.ptr(scales, "scales", _types("u8"), T * (H // 32)))


def moe_act_unpack8(codes, scales, T, H, x, x_dtype, stream=None):
    c = _Call("moe_act_unpack8")
    return c.run(stream, c.ptr(codes, "codes", _types(MOE_Q8), T * H),
                 c.ptr(scales, "scales", _types("u8"), T * (H // 32)), T, H, c.ptr(x, "x", _types(x_dtype), T * H),
                 x_dtype)


def moe_balance_ws_size(T, E):
    from . import lib
    return lib().moe_balance_ws_size(T, E)


def moe_balance_loss(logits, topk_ids, token_mask, T, E, k, balance_coef, z_coef, counts, loss, ws=None, ws_bytes=0,
                     stream=None):
    c = _Call("moe_balance_loss")
    return c.run(stream, c.ptr(logits, "logits", _types(0), T * E), c.ptr(topk_ids, "topk_ids", _types("i32"), T * k),
                 c.ptr(token_mask, "token_mask", _types("mask"), T), T, E, k, balance_coef, z_coef,
                 c.ptr(counts, "counts", _types("i32"), E + 1), c.ptr(loss, "loss", _types(0), 4),
                 c.ptr(ws, "ws", _types("u8"), ws_bytes), ws_bytes)


def moe_route_backward(logits, topk_ids, topk_w, d_topk_w, token_mask, counts, d_loss, T, E, k, balance_coef, z_coef,
                       d_logits, dl_dtype, stream=None):
    c = _Call("moe_route_backward")
    return c.run(stream, c.ptr(logits, "logits", _types(0), T * E), c.ptr(topk_ids, "topk_ids", _types("i32"), T * k),
                 c.ptr(topk_w, "topk_w", _types(0), T * k), c.ptr(d_topk_w, "d_topk_w", _types(0), T * k),
                 c.ptr(token_mask, "token_mask", _types("mask"), T), c.ptr(counts, "counts", _types("i32"), E + 1),
                 c.ptr(d_loss, "d_loss", _types(0), 1), T, E, k, balance_coef, z_coef,
                 c.ptr(d_logits, "d_logits", _types(dl_dtype), T * E), dl_dtype)


def moe_expert_ffn_backward_ws_size(bits, T, k, H, I, E, mode=0):
    from . import lib
    return lib().moe_expert_ffn_backward_ws_size(bits, T, k, H, I, E, mode)


def moe_expert_ffn_backward(bits, expert_blobs, expert_offsets, active, perm_src, perm_dst, topk_w, x, x_dtype,
                            x_scales, dy, dy_dtype, T, k, H, I, E, shared_blob, dx, dx_dtype, d_topk_w, mode=0,
                            ws=None, ws_bytes=0, stream=None):
    c = _Call("moe_expert_ffn_backward")
    i32 = _types("i32")
    blob = 3 * H * I * bits // 8 + 3 * H * I // 16
    return c.run(stream, bits, c.ptr(expert_blobs, "expert_blobs", _types("i64"), E),
                 c.ptr(expert_offsets, "expert_offsets", i32, E + 1), c.ptr(active, "active", i32, 1),
                 c.ptr(perm_src, "perm_src", i32, T * k), c.ptr(perm_dst, "perm_dst", i32, T * k),
                 c.ptr(topk_w, "topk_w", _types(0), T * k), c.ptr(x, "x", _types(x_dtype), T * H), x_dtype,
                 c.ptr(x_scales, "x_scales", _types("u8"), T * (H // 32)), c.ptr(dy, "dy", _types(dy_dtype), T * H),
                 dy_dtype, T, k, H, I, E, c.ptr(shared_blob, "shared_blob", _types("u8"), blob),
                 c.ptr(dx, "dx", _types(dx_dtype), T * H), dx_dtype, c.ptr(d_topk_w, "d_topk_w", _types(0), T * k), mode,
                 c.ptr(ws, "ws", _types("u8"), ws_bytes), ws_bytes)


def moe_router_backward_ws_size(T, H, E, dl_dtype, x_dtype, w_dtype):
    from . import lib
    return lib().moe_router_backward_ws_size(T, H, E, dl_dtype, x_dtype, w_dtype)


def moe_router_backward(d_logits, dl_dtype, x, x_dtype, w_router, w_dtype, dx_in, T, H, E, dx, dx_dtype, d_w, d_bias,
                        ws=None, ws_bytes=0, stream=None):
    c = _Call("moe_router_backward")
    return c.run(stream, c.ptr(d_logits, "d_logits", _types(dl_dtype), T * E), dl_dtype,
                 c.ptr(x, "x", _types(x_dtype), T * H), x_dtype, c.ptr(w_router, "w_router", _types(w_dtype), E * H),
                 w_dtype, c.ptr(dx_in, "dx_in", _types(0), T * H), T, H, E, c.ptr(dx, "dx", _types(dx_dtype), T * H),
                 dx_dtype, c.ptr(d_w, "d_w", _types(w_dtype), E * H), c.ptr(d_bias, "d_bias", _types(0), E),
                 c.ptr(ws, "ws", _types("u8"), ws_bytes), ws_bytes)


class TrainStep:
    """One layer's forward and backward pass over T tokens, experts frozen.

    Holds every buffer of the step, so each step that is in flight at the same
    time (a layer of a model, a micro-batch) has its own.  Between the passes
    it keeps the layer's input in 8 bits (moe_act_pack8), the logits and the
    routing; the experts' inner values are recomputed.

    layer: a MoELayer with a router; x_dtype / dy_dtype / dx_dtype: MOE_F32 or
    MOE_BF16; mode: MOE_MODE_* of both passes; balance_coef, z_coef: weights
    of the two router losses (0, 0: none are computed).
    """

    def __init__(self, layer, T, x_dtype, dy_dtype=0, dx_dtype=None, mode=0, balance_coef=0.0, z_coef=0.0):
        import torch
        from . import MOE_BF16
        from .layer import alloc_step_buffers
        if layer.w_router is None:
            raise ValueError("TrainStep needs a layer with a router")
        if T < 1:
            raise ValueError(f"T must be >= 1 (got {T})")
        self.layer, self.T, self.mode = layer, T, mode
        self.x_dtype, self.dy_dtype = x_dtype, dy_dtype
        self.dx_dtype = x_dtype if dx_dtype is None else dx_dtype
        self.balance_coef, self.z_coef = float(balance_coef), float(z_coef)
        E, H, I, k, dev = layer.E, layer.H, layer.I, layer.k, layer.device
        def new(n, dtype):
            return torch.empty(n, dtype=dtype, device=dev)
        f32, u8 = torch.float32, torch.uint8
        self.bufs = alloc_step_buffers(T, H, I, E, k, layer.bits, mode, dev, layer.shared is not None)
        self.codes, self.scales = new((T, H), torch.int8), new((T, H // 32), u8)
        self.counts, self.loss = new(E + 1, torch.int32), torch.zeros(4, dtype=f32, device=dev)
        self.mask = None
        # the router's products read the checkpoint as bf16 when its weights are bf16 (exact either way)
        self.dl_dtype = self.r_dtype = layer.w_dtype
        wide = torch.bfloat16 if layer.w_dtype == MOE_BF16 else f32
        self.x_back, self.d_logits = new((T, H), wide), new((T, E), wide)
        self.dx_experts, self.d_topk_w = new((T, H), f32), new((T, k), f32)
        self.dx = new((T, H), torch.bfloat16 if self.dx_dtype == MOE_BF16 else f32)
        self.d_w_router, self.d_bias = torch.empty_like(layer.w_router), new(E, f32)
        self.sizes = dict(balance=moe_balance_ws_size(T, E),
                          ffn=moe_expert_ffn_backward_ws_size(layer.bits, T, k, H, I, E, mode),
                          router=moe_router_backward_ws_size(T, H, E, self.dl_dtype, self.r_dtype, layer.w_dtype))
        self.ws = new(max(16, *self.sizes.values()), u8)
        self._ran = False

    def forward(self, x, token_mask=None, stream=None):
        """x: device [T, H] (x_dtype); token_mask: device uint8/bool [T], 0 for
        padding (kept for the backward pass), or None.  Returns (y, loss): y
        fp32 [T, H], loss fp32 [4] = total, balance, z, counted tokens."""
        L, T, b = self.layer, self.T, self.bufs
        L.forward(x, self.x_dtype, T=T, mode=self.mode, stream=stream, bufs=b)
        moe_act_pack8(x, self.x_dtype, T, L.H, self.codes, self.scales, stream)
        self.mask = token_mask
        if self.balance_coef or self.z_coef:
            moe_balance_loss(b.logits, b.ids, token_mask, T, L.E, L.k, self.balance_coef, self.z_coef, self.counts,
                             self.loss, self.ws, self.sizes["balance"], stream)
        self._ran = True
        return b.y[:T * L.H].view(T, L.H), self.loss

    def backward(self, dy, d_loss=None, stream=None):
        """dy: device [T, H] (dy_dtype), the gradient of y; rows of masked
        tokens must be zero.  d_loss: device fp32 scalar, the gradient of
        loss[0] (None: 1).  Returns dict(dx, d_w_router, d_bias), buffers of
        this object that the next backward() overwrites."""
        if not self._ran:
            raise RuntimeError("TrainStep.backward() needs a forward() first")
        L, T, b = self.layer, self.T, self.bufs
        E, H, I, k = L.E, L.H, L.I, L.k
        loss = bool(self.balance_coef or self.z_coef)
        moe_expert_ffn_backward(L.bits, L.table, b.offsets, b.active, b.perm_src, b.perm_dst, b.w, self.codes, MOE_Q8,
                                self.scales, dy, self.dy_dtype, T, k, H, I, E, L.shared, self.dx_experts, 0,
                                self.d_topk_w, self.mode, self.ws, self.sizes["ffn"], stream)
        moe_route_backward(b.logits, b.ids, b.w, self.d_topk_w, self.mask, self.counts if loss else None, d_loss, T,
                           E, k, self.balance_coef, self.z_coef, self.d_logits, self.dl_dtype, stream)
        moe_act_unpack8(self.codes, self.scales, T, H, self.x_back, self.r_dtype, stream)
        moe_router_backward(self.d_logits, self.dl_dtype, self.x_back, self.r_dtype, L.w_router, L.w_dtype,
                            self.dx_experts, T, H, E, self.dx, self.dx_dtype, self.d_w_router, self.d_bias, self.ws,
                            self.sizes["router"], stream)
        return dict(dx=self.dx, d_w_router=self.d_w_router, d_bias=self.d_bias)
