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

_PTR, _INT, _FLT, _SZ = C.c_void_p, C.c_int, C.c_float, C.c_size_t
SIGNATURES = {
    "moe_act_pack8": (_INT, [_PTR, _INT, _INT, _INT, _PTR, _PTR, _PTR]),
    "moe_act_unpack8": (_INT, [_PTR, _PTR, _INT, _INT, _PTR, _INT, _PTR]),
    "moe_balance_ws_size": (_SZ, [_INT, _INT]),
    "moe_balance_loss": (_INT, [_PTR, _PTR, _PTR, _INT, _INT, _INT, _FLT, _FLT, _PTR, _PTR, _PTR, _SZ, _PTR]),
    "moe_route_backward": (_INT, [_PTR, _PTR, _PTR, _PTR, _PTR, _PTR, _PTR, _INT, _INT, _INT, _FLT, _FLT, _PTR, _INT,
                                  _PTR]),
    "moe_expert_ffn_backward_ws_size": (_SZ, [_INT, _INT, _INT, _INT, _INT, _INT, _INT]),
    "moe_expert_ffn_backward": (_INT, [_INT, _PTR, _PTR, _PTR, _PTR, _PTR, _PTR, _PTR, _INT, _PTR, _PTR, _INT, _INT,
                                       _INT, _INT, _INT, _INT, _PTR, _PTR, _INT, _PTR, _INT, _PTR, _SZ, _PTR]),
    "moe_router_backward_ws_size": (_SZ, [_INT, _INT, _INT, _INT, _INT, _INT]),
    "moe_router_backward": (_INT, [_PTR, _INT, _PTR, _INT, _PTR, _INT, _PTR, _INT, _INT, _INT, _PTR, _INT, _PTR, _PTR,
                                   _PTR, _SZ, _PTR]),
}


# A call's checks and marshalling are most of a small call's time on the host:
# the good case of _p is five attribute reads, and everything that can be looked
# up once is.
_lib = _current = _raw_stream = None        # the library; the current device; a device's current stream
_T = {}                                     # dtype code -> torch types


def _load():
    """First call: the library and what the checks need of torch."""
    global _lib, _current, _raw_stream
    import torch
    from . import lib
    f32, bf16, i8 = torch.float32, torch.bfloat16, torch.int8
    _T.update({0: (f32,), 1: (bf16,), MOE_Q8: (i8,), "i32": (torch.int32,), "i64": (torch.int64,),
               "u8": (torch.uint8,), "mask": (torch.uint8, torch.bool), None: (f32, bf16, i8)})
    _current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: torch.cuda.current_stream(d).cuda_stream)
    _lib = lib()
    return _lib


def _any(code):
    """torch types of a dtype argument (an unknown code passes: the C call refuses it)."""
    return _T.get(code) or _T[None]


def _p(dev, name, what, t, types, count):
    """(device, pointer) of a buffer of at least `count` values of one of `types`;
    None and addresses pass.  dev: the device of the buffers before it, or None."""
    if t is None:
        return dev, None
    try:
        d = t.get_device()
        if t.dtype in types and (d == dev or dev is None) and d >= 0 and t.is_contiguous() and t.numel() >= count:
            return d, t.data_ptr()
    except AttributeError:
        pass
    if isinstance(t, int):
        return dev, t
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: {what} must be a CUDA tensor, an address or None (got {type(t).__name__})")
    if not t.is_cuda:
        raise ValueError(f"{name}: {what} must be a CUDA tensor (got {t.device})")
    if t.dtype not in types:
        raise ValueError(f"{name}: {what} has type {t.dtype}, expected {' or '.join(map(str, types))}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: {what} must be contiguous")
    if t.numel() < count:
        raise ValueError(f"{name}: {what} holds {t.numel()} values, needs {count}")
    raise ValueError(f"{name}: {what} is on {t.device}, other buffers on cuda:{dev}")


def _run(fn, dev, stream, *args):
    """Calls fn(*args, stream) on the buffers' device."""
    here = _current()
    if dev is None or dev == here:
        rc = fn(*args, _raw_stream(here) if stream is None else getattr(stream, "cuda_stream", stream))
    else:
        import torch
        with torch.cuda.device(dev):
            rc = fn(*args, _raw_stream(dev) if stream is None else getattr(stream, "cuda_stream", stream))
    if rc:
        from . import _check
        _check(rc)
    return rc


def moe_act_pack8(x, x_dtype, T, H, codes, scales, stream=None):
    f = (_lib or _load()).moe_act_pack8
    n = "moe_act_pack8"
    d, x = _p(None, n, "x", x, _any(x_dtype), T * H)
    d, codes = _p(d, n, "codes", codes, _T[MOE_Q8], T * H)
    d, scales = _p(d, n, "scales", scales, _T["u8"], T * (H // 32))
    return _run(f, d, stream, x, x_dtype, T, H, codes, scales)


def moe_act_unpack8(codes, scales, T, H, x, x_dtype, stream=None):
    f = (_lib or _load()).moe_act_unpack8
    n = "moe_act_unpack8"
    d, codes = _p(None, n, "codes", codes, _T[MOE_Q8], T * H)
    d, scales = _p(d, n, "scales", scales, _T["u8"], T * (H // 32))
    d, x = _p(d, n, "x", x, _any(x_dtype), T * H)
    return _run(f, d, stream, codes, scales, T, H, x, x_dtype)


def moe_balance_ws_size(T, E):
    return (_lib or _load()).moe_balance_ws_size(T, E)


def moe_balance_loss(logits, topk_ids, token_mask, T, E, k, balance_coef, z_coef, counts, loss, ws=None, ws_bytes=0,
                     stream=None):
    f = (_lib or _load()).moe_balance_loss
    n = "moe_balance_loss"
    d, logits = _p(None, n, "logits", logits, _T[0], T * E)
    d, topk_ids = _p(d, n, "topk_ids", topk_ids, _T["i32"], T * k)
    d, token_mask = _p(d, n, "token_mask", token_mask, _T["mask"], T)
    d, counts = _p(d, n, "counts", counts, _T["i32"], E + 1)
    d, loss = _p(d, n, "loss", loss, _T[0], 4)
    d, ws = _p(d, n, "ws", ws, _T["u8"], ws_bytes)
    return _run(f, d, stream, logits, topk_ids, token_mask, T, E, k, balance_coef, z_coef, counts, loss, ws, ws_bytes)


def moe_route_backward(logits, topk_ids, topk_w, d_topk_w, token_mask, counts, d_loss, T, E, k, balance_coef, z_coef,
                       d_logits, dl_dtype, stream=None):
    f = (_lib or _load()).moe_route_backward
    n = "moe_route_backward"
    d, logits = _p(None, n, "logits", logits, _T[0], T * E)
    d, topk_ids = _p(d, n, "topk_ids", topk_ids, _T["i32"], T * k)
    d, topk_w = _p(d, n, "topk_w", topk_w, _T[0], T * k)
    d, d_topk_w = _p(d, n, "d_topk_w", d_topk_w, _T[0], T * k)
    d, token_mask = _p(d, n, "token_mask", token_mask, _T["mask"], T)
    d, counts = _p(d, n, "counts", counts, _T["i32"], E + 1)
    d, d_loss = _p(d, n, "d_loss", d_loss, _T[0], 1)
    d, d_logits = _p(d, n, "d_logits", d_logits, _any(dl_dtype), T * E)
    return _run(f, d, stream, logits, topk_ids, topk_w, d_topk_w, token_mask, counts, d_loss, T, E, k, balance_coef,
                z_coef, d_logits, dl_dtype)


def moe_expert_ffn_backward_ws_size(bits, T, k, H, I, E, mode=0):
    return (_lib or _load()).moe_expert_ffn_backward_ws_size(bits, T, k, H, I, E, mode)


def moe_expert_ffn_backward(bits, expert_blobs, expert_offsets, active, perm_src, perm_dst, topk_w, x, x_dtype,
                            x_scales, dy, dy_dtype, T, k, H, I, E, shared_blob, dx, dx_dtype, d_topk_w, mode=0,
                            ws=None, ws_bytes=0, stream=None):
    f = (_lib or _load()).moe_expert_ffn_backward
    n, i32 = "moe_expert_ffn_backward", _T["i32"]
    d, expert_blobs = _p(None, n, "expert_blobs", expert_blobs, _T["i64"], E)
    d, expert_offsets = _p(d, n, "expert_offsets", expert_offsets, i32, E + 1)
    d, active = _p(d, n, "active", active, i32, 1)
    d, perm_src = _p(d, n, "perm_src", perm_src, i32, T * k)
    d, perm_dst = _p(d, n, "perm_dst", perm_dst, i32, T * k)
    d, topk_w = _p(d, n, "topk_w", topk_w, _T[0], T * k)
    d, x = _p(d, n, "x", x, _any(x_dtype), T * H)
    d, x_scales = _p(d, n, "x_scales", x_scales, _T["u8"], T * (H // 32))
    d, dy = _p(d, n, "dy", dy, _any(dy_dtype), T * H)
    d, shared_blob = _p(d, n, "shared_blob", shared_blob, _T["u8"], 3 * H * I * bits // 8 + 3 * H * I // 16)
    d, dx = _p(d, n, "dx", dx, _any(dx_dtype), T * H)
    d, d_topk_w = _p(d, n, "d_topk_w", d_topk_w, _T[0], T * k)
    d, ws = _p(d, n, "ws", ws, _T["u8"], ws_bytes)
    return _run(f, d, stream, bits, expert_blobs, expert_offsets, active, perm_src, perm_dst, topk_w, x, x_dtype,
                x_scales, dy, dy_dtype, T, k, H, I, E, shared_blob, dx, dx_dtype, d_topk_w, mode, ws, ws_bytes)


def moe_router_backward_ws_size(T, H, E, dl_dtype, x_dtype, w_dtype):
    return (_lib or _load()).moe_router_backward_ws_size(T, H, E, dl_dtype, x_dtype, w_dtype)


def moe_router_backward(d_logits, dl_dtype, x, x_dtype, w_router, w_dtype, dx_in, T, H, E, dx, dx_dtype, d_w, d_bias,
                        ws=None, ws_bytes=0, stream=None):
    f = (_lib or _load()).moe_router_backward
    n = "moe_router_backward"
    d, d_logits = _p(None, n, "d_logits", d_logits, _any(dl_dtype), T * E)
    d, x = _p(d, n, "x", x, _any(x_dtype), T * H)
    d, w_router = _p(d, n, "w_router", w_router, _any(w_dtype), E * H)
    d, dx_in = _p(d, n, "dx_in", dx_in, _T[0], T * H)
    d, dx = _p(d, n, "dx", dx, _any(dx_dtype), T * H)
    d, d_w = _p(d, n, "d_w", d_w, _any(w_dtype), E * H)
    d, d_bias = _p(d, n, "d_bias", d_bias, _T[0], E)
    d, ws = _p(d, n, "ws", ws, _T["u8"], ws_bytes)
    return _run(f, d, stream, d_logits, dl_dtype, x, x_dtype, w_router, w_dtype, dx_in, T, H, E, dx, dx_dtype, d_w,
                d_bias, ws, ws_bytes)


class TrainStep:
    """One layer's forward and backward pass over T tokens, experts frozen.

    Holds every buffer of the step, so each step that is in flight at the same
    time (a layer of a model, a micro-batch) has its own.  Between the passes
    it keeps the layer's input in 8 bits (moe_act_pack8), the logits and the
    routing; the experts' inner values are recomputed.

    layer: a MoELayer with a router; x_dtype / dy_dtype / dx_dtype: MOE_F32 or
    MOE_BF16; mode: MOE_MODE_* of both passes; balance_coef, z_coef: weights
    of the two router losses (0, 0: none are computed).

    The gradient of the logits is kept in the type of the router's weights
    (rounded once; bf16: half a step is 2^-8 of a value), since the router's
    tensor-core products take bf16 operands only, and d_w_router has that type
    too: a router whose gradient is wanted in fp32 is one with w_dtype "f32".
    Of what a step holds only the checkpoint, the logits and the routing live
    from forward() to backward(): 35 MB of 2.1 GB at 8192 tokens through
    top-10 of 512 experts of 2048 x 512; the rest is scratch of its own.
    """

    def __init__(self, layer, T, x_dtype, dy_dtype=0, dx_dtype=None, mode=0, balance_coef=0.0, z_coef=0.0):
        import torch
        if layer.w_router is None:
            raise ValueError("TrainStep needs a layer with a router")
        if T < 1:
            raise ValueError(f"T must be >= 1 (got {T})")
        self.layer, self.T, self.mode = layer, T, mode
        self.x_dtype, self.dy_dtype = x_dtype, dy_dtype
        self.dx_dtype = x_dtype if dx_dtype is None else dx_dtype
        self.balance_coef, self.z_coef = float(balance_coef), float(z_coef)
        self.device = layer.arena.device                # layer.device may have no index
        with torch.cuda.device(self.device):            # sizes follow the current device
            self._allocate()
        self.mask = None
        self._ran = False

    def _allocate(self):
        import torch
        from . import MOE_BF16
        from .layer import alloc_step_buffers
        layer, T, mode, dev = self.layer, self.T, self.mode, self.device
        E, H, I, k = layer.E, layer.H, layer.I, layer.k

        def new(n, dtype):
            return torch.empty(n, dtype=dtype, device=dev)
        f32, u8 = torch.float32, torch.uint8
        self.bufs = alloc_step_buffers(T, H, I, E, k, layer.bits, mode, dev, layer.shared is not None)
        self.codes, self.scales = new((T, H), torch.int8), new((T, H // 32), u8)
        self.counts, self.loss = new(E + 1, torch.int32), torch.zeros(4, dtype=f32, device=dev)
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

    def forward(self, x, token_mask=None, stream=None):
        """x: device [T, H] (x_dtype); token_mask: device uint8/bool [T], 0 for
        padding (kept for the backward pass), or None; rows of padding have to
        be finite, since they go through the layer like the others.  Returns
        (y, loss): y fp32 [T, H], loss fp32 [4] = total, balance, z, counted
        tokens.  Arguments are checked before anything is launched; after an
        error there is no backward() until a forward() has succeeded."""
        import torch
        self._ran = False                               # the buffers below belong to no whole step until the end
        L, T, b, n = self.layer, self.T, self.bufs, "TrainStep.forward"
        d, _ = _p(self.device.index, n, "x", x, _any(self.x_dtype), T * L.H)
        _p(d, n, "token_mask", token_mask, _T["mask"], T)
        with torch.cuda.device(self.device):            # the forward calls run on the current device
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
        d, _ = _p(self.device.index, "TrainStep.backward", "dy", dy, _any(self.dy_dtype), T * H)
        _p(d, "TrainStep.backward", "d_loss", d_loss, _T[0], 1)
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
