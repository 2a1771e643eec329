"""Timed cases of the expert step's backward side.

Four operators that train around frozen quantized experts: 8-bit activation
checkpoints, the balance loss with its gradient, the quantized experts'
backward pass from a checkpoint, and the router's products.  Each has a plain
form in elementary torch operations (own = False) and the library's calls
(own = True).  Sizes are the ones of the repository's workloads (hidden 2048,
intermediate 512, 512 experts, top-10, chunks up to 8192 tokens; 256 x 128
with 16 experts, top-2, for the smallest) and generic ragged ones.
"""
import math

import torch

own = False

BLOCK = 32


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token's activation kept for a later backward pass
        {"name": "checkpoint token", "op": "checkpoint", "T": 1, "H": 2048, "dtype": "bf16"},
        # a ragged batch of fp32 activations
        {"name": "checkpoint ragged f32", "op": "checkpoint", "T": 777, "H": 1184, "dtype": "f32"},
        # the largest prompt chunk
        {"name": "checkpoint chunk", "op": "checkpoint", "T": 8192, "H": 2048, "dtype": "bf16"},
        # the smallest router: 8 tokens over 16 experts
        {"name": "balance small", "op": "balance", "T": 8, "E": 16, "k": 2, "masked": 0.0, "dtype": "f32"},
        # a padded training batch over one layer's experts
        {"name": "balance chunk", "op": "balance", "T": 8192, "E": 512, "k": 10, "masked": 0.1, "dtype": "f32"},
        # one model-wide pool of experts
        {"name": "balance pool", "op": "balance", "T": 129, "E": 24576, "k": 10, "masked": 0.0, "dtype": "bf16"},
        # one token's gradient (online adaptation while decoding)
        {"name": "experts token", "op": "experts", "bits": 4, "T": 1, "H": 2048, "I": 512, "E": 512, "k": 10,
         "shared": True, "dy": "f32"},
        # a short window through 2-bit experts
        {"name": "experts window 2-bit", "op": "experts", "bits": 2, "T": 16, "H": 2048, "I": 512, "E": 512, "k": 10,
         "shared": True, "dy": "bf16"},
        # a ragged batch, few experts, no shared expert
        {"name": "experts ragged", "op": "experts", "bits": 4, "T": 777, "H": 1152, "I": 384, "E": 40, "k": 3,
         "shared": False, "dy": "f32"},
        # a training batch of the largest chunk
        {"name": "experts chunk", "op": "experts", "bits": 4, "T": 8192, "H": 2048, "I": 512, "E": 512, "k": 10,
         "shared": True, "dy": "bf16"},
        # the router's gradients of a small batch
        {"name": "router window", "op": "router", "T": 33, "H": 2048, "E": 512},
        # and of the largest chunk
        {"name": "router chunk", "op": "router", "T": 8192, "H": 2048, "E": 512},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["checkpoint", "balance", "experts", "experts", "router"])
    if op == "checkpoint":
        H = 32 * _log_int(rng, 1, 128)
        return {"op": op, "T": _log_int(rng, 1, min(8192, (8192 * 2048) // H)), "H": H,
                "dtype": rng.choice(["bf16", "f32"])}
    if op == "balance":
        E = _log_int(rng, 8, 24576)
        return {"op": op, "T": _log_int(rng, 1, max(1, min(8192, (8192 * 512) // E))), "E": E,
                "k": rng.randint(1, min(E, 16)), "masked": rng.choice([0.0, 0.1, 0.5]),
                "dtype": rng.choice(["f32", "bf16"])}
    if op == "experts":
        E = _log_int(rng, 8, 512)
        return {"op": op, "bits": rng.choice([2, 4]), "T": _log_int(rng, 1, 4096), "H": 128 * rng.randint(1, 16),
                "I": 128 * rng.randint(1, 4), "E": E, "k": rng.randint(1, min(E, 10)),
                "shared": rng.choice([False, True]), "dy": rng.choice(["f32", "bf16"])}
    return {"op": op, "T": _log_int(rng, 1, 8192), "H": 8 * _log_int(rng, 16, 256), "E": 8 * _log_int(rng, 1, 64)}


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _size(name):
    return 2 if name == "bf16" else 4


# ------------------------------------------------------------------ inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, T, H):
    """Hidden states: unit normal, each token with its own level."""
    return _normal(g, T, H) * torch.exp(0.3 * _normal(g, T, 1))


def _steps(x):
    """The 8-bit checkpoint of x: (whole codes, step per block of 32) as fp32."""
    b = x.float().reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1)
    e = torch.frexp(amax)[1] - 7
    e = torch.where(amax == 0, torch.full_like(e, -126), e).clamp(-126, 127)
    inv = ((127 - e) << 23).view(torch.float32)
    e = e + (torch.round(amax * inv) > 127).to(e.dtype)
    step = ((127 + e) << 23).view(torch.float32)
    inv = ((127 - e) << 23).view(torch.float32)
    q = torch.round(b * inv[..., None])
    bad = ~torch.isfinite(amax)
    return torch.where(bad[..., None], torch.zeros_like(q), q), torch.where(bad, torch.full_like(step, math.nan), step)


def _pack_matrices(w, bits):
    """[n, rows, cols] fp32 -> (codes uint8, fp16 steps) of the expert blob: the
    element of largest magnitude of each block of 32 gets the lowest code; steps
    keep 8 significant bits."""
    half = 1 << (bits - 1)
    b = w.reshape(w.shape[0], w.shape[1], -1, BLOCK)
    m = torch.gather(b, -1, b.abs().argmax(-1, keepdim=True))
    d = (m / -half).bfloat16().half()
    q = (torch.round(b / d.float()).clamp(-half, half - 1) + half).to(torch.uint8)
    if bits == 4:
        codes = q[..., :16] | (q[..., 16:] << 4)
    else:
        c = q.reshape(*q.shape[:-1], 4, 8)
        codes = c[..., 0, :] | (c[..., 1, :] << 2) | (c[..., 2, :] << 4) | (c[..., 3, :] << 6)
    return codes.reshape(w.shape[0], -1), d.reshape(w.shape[0], -1).contiguous().view(torch.uint8)


def _blobs(g, n, bits, H, I):
    out = []
    for i in range(0, n, 32):
        m = min(32, n - i)
        parts = [_pack_matrices(0.02 * _normal(g, m, r, c), bits) for r, c in ((I, H), (I, H), (H, I))]
        out.append(torch.cat([p[0] for p in parts] + [p[1] for p in parts], 1))
    return torch.cat(out)


def _routing(g, T, E, k):
    """Router logits with a mild preference of the router for some experts."""
    logits = _normal(g, T, E) + 0.2 * _normal(g, E)
    top, ids = torch.topk(logits, k, dim=1)
    return logits, ids.int(), torch.softmax(top, 1)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "checkpoint":
        T, H = case["T"], case["H"]
        st = {"x": _activations(g, T, H).to(_dtype(case["dtype"]))}
        if own:
            st["codes"] = torch.empty(T, H, dtype=torch.int8, device="cuda")
            st["scales"] = torch.empty(T, H // BLOCK, dtype=torch.uint8, device="cuda")
            st["y"] = torch.empty_like(st["x"])
    elif op == "balance":
        T, E, k = case["T"], case["E"], case["k"]
        logits, ids, w = _routing(g, T, E, k)
        mask = torch.rand(T, generator=g, device="cuda") >= case["masked"]
        st = {"logits": logits, "ids": ids, "w": w, "dw": _normal(g, T, k), "mask": mask.to(torch.uint8),
              "d_loss": torch.full((1,), 1.0, device="cuda"), "balance": 0.01 * T, "z": 0.001 * T}
        if own:
            import quantized_expert_ffn_route_b200 as M
            n = M.moe_balance_ws_size(T, E)
            st.update(counts=torch.empty(E + 1, dtype=torch.int32, device="cuda"), ws_bytes=n,
                      loss=torch.empty(4, device="cuda"), ws=torch.empty(max(16, n), dtype=torch.uint8, device="cuda"),
                      dl=torch.empty(T, E, dtype=_dtype(case["dtype"]), device="cuda"))
    elif op == "experts":
        st = _prepare_experts(case, g)
    else:
        T, H, E = case["T"], case["H"], case["E"]
        st = {"dl": (_normal(g, T, E) / 64).bfloat16(), "x": _activations(g, T, H).bfloat16(),
              "w": (0.1 * _normal(g, E, H)).bfloat16(), "dx_in": 0.01 * _normal(g, T, H)}
        if own:
            import quantized_expert_ffn_route_b200 as M
            n = M.moe_router_backward_ws_size(T, H, E, M.MOE_BF16, M.MOE_BF16, M.MOE_BF16)
            st.update(dx=torch.empty_like(st["x"]), d_w=torch.empty_like(st["w"]),
                      d_bias=torch.empty(E, device="cuda"), ws_bytes=n,
                      ws=torch.empty(max(16, n), dtype=torch.uint8, device="cuda"))
    st["case"] = dict(case)
    return st


def _prepare_experts(case, g):
    bits, T, H, I, E, k = (case[n] for n in ("bits", "T", "H", "I", "E", "k"))
    blobs = _blobs(g, E + 1, bits, H, I)
    q, step = _steps(_activations(g, T, H))
    logits, ids, w = _routing(g, T, E, k)
    st = {"blobs": blobs[:E], "shared": blobs[E] if case["shared"] else None, "logits": logits, "ids": ids, "w": w,
          "codes": q.reshape(T, H).to(torch.int8), "scales": (torch.frexp(step)[1] + 126).to(torch.uint8),
          "dy": (_normal(g, T, H) / 1024).to(_dtype(case["dy"]))}
    # the permutation that the forward pass left: rows grouped by expert, tokens ascending
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True)[1]
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    perm_dst = torch.empty_like(order)
    perm_dst[order] = torch.arange(T * k, device="cuda")
    live = torch.nonzero(counts).reshape(-1)
    st.update(offsets=offsets.int(), perm_src=(order // k).int(), perm_dst=perm_dst.int(),
              active=torch.cat([torch.tensor([live.numel()], device="cuda"), live]).int())
    # the same rows as a padded batch of the experts in use: row numbers, T*k where there is none
    most = int(counts.max())
    at = offsets[live][:, None] + torch.arange(most, device="cuda")
    st.update(live=live, rows=torch.where(at < offsets[live + 1][:, None], at, torch.full_like(at, T * k)))
    if own:
        import quantized_expert_ffn_route_b200 as M
        n = M.moe_expert_ffn_backward_ws_size(bits, T, k, H, I, E, M.MOE_MODE_AUTO)
        st.update(layer=M.MoELayer(bits, H, I, E, k, st["blobs"], None if st["shared"] is None else st["shared"].cpu()),
                  dx=torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), dw=torch.empty(T, k, device="cuda"),
                  dl=torch.empty(T, E, dtype=torch.bfloat16, device="cuda"), ws_bytes=n,
                  ws=torch.empty(max(16, n), dtype=torch.uint8, device="cuda"))
    return st


# ------------------------------------------------------------- plain forms
def _plain_checkpoint(st):
    q, step = _steps(st["x"])
    return {"x": (q * step[..., None]).reshape(st["x"].shape).to(st["x"].dtype)}


def _plain_route_backward(logits, ids, w, dw, valid, counts, g, balance, z):
    T, E = logits.shape
    k = ids.shape[1]
    n = valid.sum().clamp(min=1).float()
    m = logits.amax(1, keepdim=True)
    p = torch.exp(logits - m)
    s = p.sum(1, keepdim=True)
    p, lse = p / s, m + torch.log(s)
    f = counts.float() / (n * k)
    dl = g * p * (balance * E / n * (f - (f * p).sum(1, keepdim=True)) + z * 2 * lse / n)
    dl.scatter_add_(1, ids.long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return torch.where(valid[:, None], dl, torch.zeros_like(dl)), p, lse, f, n


def _plain_balance(st):
    case = st["case"]
    valid = st["mask"] != 0
    k, E = case["k"], case["E"]
    counts = torch.zeros(E, dtype=torch.int32, device="cuda")
    counts.scatter_add_(0, st["ids"].reshape(-1).long(), valid[:, None].expand(-1, k).reshape(-1).int())
    dl, p, lse, f, n = _plain_route_backward(st["logits"], st["ids"], st["w"], st["dw"], valid, counts, st["d_loss"],
                                             st["balance"], st["z"])
    balance = E * (f * torch.where(valid[:, None], p, torch.zeros_like(p)).double().sum(0).float() / n).sum()
    z = torch.where(valid, lse[:, 0] * lse[:, 0], torch.zeros_like(lse[:, 0])).double().sum().float() / n
    loss = torch.stack([st["balance"] * balance + st["z"] * z, balance, z])
    return {"loss": loss, "counts": counts, "d_logits": dl.to(_dtype(case["dtype"]))}


def _weights(blobs, bits, H, I):
    """The three matrices of each blob in fp32: gate and up [n, I, H], down [n, H, I]."""
    n, nb = blobs.shape[0], I * H * bits // 8
    d = blobs[:, 3 * nb:].contiguous().view(torch.float16).float().reshape(n, 3, -1)
    c = blobs[:, :3 * nb].reshape(n, 3, -1, 4 * bits)
    if bits == 4:
        q = torch.cat([c & 15, c >> 4], -1)
    else:
        q = torch.cat([c & 3, (c >> 2) & 3, (c >> 4) & 3, c >> 6], -1)
    w = ((q.float() - (1 << (bits - 1))) * d[..., None]).reshape(n, 3, -1)
    return w[:, 0].reshape(n, I, H), w[:, 1].reshape(n, I, H), w[:, 2].reshape(n, H, I)


def _plain_ffn_backward(wg, wu, wd, x, dy):
    """[n, tokens, H] inputs -> (dx, <dy, y>) of each expert's tokens."""
    g, u, q = x @ wg.transpose(1, 2), x @ wu.transpose(1, 2), dy @ wd
    s = 1 / (1 + torch.exp(-g))
    a = g * s
    dx = (q * u * (s + a * (1 - s))) @ wg + (q * a) @ wu
    return dx, (q * a * u).sum(-1)


def _plain_experts(st):
    case = st["case"]
    bits, T, H, I, E, k = (case[n] for n in ("bits", "T", "H", "I", "E", "k"))
    step = ((st["scales"].int()) << 23).view(torch.float32)
    x = (st["codes"].float().reshape(T, -1, BLOCK) * step[..., None]).reshape(T, H)
    dy = st["dy"].float()
    src = torch.cat([st["perm_src"].long(), torch.zeros(1, dtype=torch.int64, device="cuda")])[st["rows"]]
    dxp, dwp = _plain_ffn_backward(*_weights(st["blobs"][st["live"]], bits, H, I), x[src], dy[src])
    rows = torch.zeros(T * k + 1, H, device="cuda")
    rows[st["rows"].reshape(-1)] = dxp.reshape(-1, H)
    gates = torch.zeros(T * k + 1, device="cuda")
    gates[st["rows"].reshape(-1)] = dwp.reshape(-1)
    dst = st["perm_dst"].long().reshape(T, k)
    dx = (st["w"][..., None] * rows[dst]).sum(1)
    if st["shared"] is not None:
        dx = dx + _plain_ffn_backward(*_weights(st["shared"][None], bits, H, I), x[None], dy[None])[0][0]
    valid = torch.ones(T, dtype=torch.bool, device="cuda")
    dl = _plain_route_backward(st["logits"], st["ids"], st["w"], gates[dst], valid,
                               torch.zeros(E, device="cuda"), 0.0, 0.0, 0.0)[0]
    return {"dx": dx.bfloat16(), "d_logits": dl.bfloat16()}


def _plain_router(st):
    dl, x, w = st["dl"].float(), st["x"].float(), st["w"].float()
    return {"dx": (st["dx_in"] + dl @ w).bfloat16(), "d_w": (dl.t() @ x).bfloat16(), "d_bias": dl.sum(0)}


# --------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "checkpoint":
            return _plain_checkpoint(state)
        if op == "balance":
            return _plain_balance(state)
        if op == "experts":
            return _plain_experts(state)
        return _plain_router(state)
    import quantized_expert_ffn_route_b200 as M
    c, st = state["case"], state
    T = c["T"]
    if op == "checkpoint":
        dt = M.MOE_BF16 if c["dtype"] == "bf16" else M.MOE_F32
        M.moe_act_pack8(st["x"], dt, T, c["H"], st["codes"], st["scales"])
        M.moe_act_unpack8(st["codes"], st["scales"], T, c["H"], st["y"], dt)
        return {"x": st["y"]}
    if op == "balance":
        E, k = c["E"], c["k"]
        M.moe_balance_loss(st["logits"], st["ids"], st["mask"], T, E, k, st["balance"], st["z"], st["counts"],
                           st["loss"], st["ws"], st["ws_bytes"])
        M.moe_route_backward(st["logits"], st["ids"], st["w"], st["dw"], st["mask"], st["counts"], st["d_loss"], T, E,
                             k, st["balance"], st["z"], st["dl"], M.MOE_BF16 if c["dtype"] == "bf16" else M.MOE_F32)
        return {"loss": st["loss"][:3], "counts": st["counts"][:E], "d_logits": st["dl"]}
    if op == "experts":
        bits, H, I, E, k = (c[n] for n in ("bits", "H", "I", "E", "k"))
        layer = st["layer"]
        M.moe_expert_ffn_backward(bits, layer.table, st["offsets"], st["active"], st["perm_src"], st["perm_dst"],
                                  st["w"], st["codes"], M.MOE_Q8, st["scales"], st["dy"],
                                  M.MOE_BF16 if c["dy"] == "bf16" else M.MOE_F32, T, k, H, I, E, layer.shared,
                                  st["dx"], M.MOE_BF16, st["dw"], M.MOE_MODE_AUTO, st["ws"], st["ws_bytes"])
        M.moe_route_backward(st["logits"], st["ids"], st["w"], st["dw"], None, None, None, T, E, k, 0.0, 0.0,
                             st["dl"], M.MOE_BF16)
        return {"dx": st["dx"], "d_logits": st["dl"]}
    M.moe_router_backward(st["dl"], M.MOE_BF16, st["x"], M.MOE_BF16, st["w"], M.MOE_BF16, st["dx_in"], T, c["H"],
                          c["E"], st["dx"], M.MOE_BF16, st["d_w"], st["d_bias"], st["ws"], st["ws_bytes"])
    return {"dx": st["dx"], "d_w": st["d_w"], "d_bias": st["d_bias"]}


# -------------------------------------------------------------------- work
def work(case):
    T = case["T"]
    if case["op"] == "checkpoint":
        n = T * case["H"]
        # read, write codes and steps, read them back, write: a handful of operations a value
        return {"bytes": n * (2 * _size(case["dtype"]) + 2 * (1 + 1 / BLOCK)), "flops": 6 * n}
    if case["op"] == "balance":
        E, k = case["E"], case["k"]
        # logits in, gradient out, ids, gates and their gradients
        return {"bytes": T * E * (4 + _size(case["dtype"])) + 12 * T * k + T + 4 * E, "flops": 12 * T * E}
    if case["op"] == "experts":
        bits, H, I, E, k = (case[n] for n in ("bits", "H", "I", "E", "k"))
        blob = 3 * H * I * bits // 8 + 3 * H * I // BLOCK * 2
        used = E * (1 - (1 - k / E) ** T) + (1 if case["shared"] else 0)
        # blobs in use, checkpoint, dy, dx; logits' gradient, routing
        nbytes = used * blob + T * H * (1 + 1 / BLOCK + _size(case["dy"]) + 2) + T * (2 * E + 16 * k)
        return {"bytes": nbytes, "flops": 10 * H * I * T * (k + (1 if case["shared"] else 0))}
    H, E = case["H"], case["E"]
    return {"bytes": 2 * (T * E + 2 * T * H + 2 * E * H) + 4 * T * H + 4 * E, "flops": 4 * T * E * H}


# ------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "checkpoint":
        x = st["x"].double().reshape(-1, BLOCK)
        top = x.abs().max(1).values
        # the smallest power of two that leaves no code above 127
        e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 6
        e = torch.where(torch.round(top * 2.0 ** -e) > 127, e + 1, e)
        e = torch.where(top > 0, e, torch.full_like(e, -126.0)).clamp(min=-126)[:, None]
        return {"x": (torch.round(x * 2.0 ** -e) * 2.0 ** e).reshape(st["x"].shape)}
    if op == "balance":
        return _exact_balance(st, case)
    if op == "experts":
        return _exact_experts(st, case)
    dl, x, w = (st[n].double() for n in ("dl", "x", "w"))
    return {"dx": torch.einsum("te,eh->th", dl, w) + st["dx_in"], "d_w": torch.einsum("te,th->eh", dl, x),
            "d_bias": torch.einsum("te->e", dl)}


def _exact_balance(st, case):
    E, k = case["E"], case["k"]
    keep = torch.nonzero(st["mask"]).reshape(-1)
    l, ids, w, dw = (st[n][keep] for n in ("logits", "ids", "w", "dw"))
    l, n = l.double(), max(1, keep.numel())
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)
    share = counts.double() / (n * k)
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    balance, z = E * torch.dot(share, p.sum(0) / n), lse.square().sum() / n
    g = torch.zeros_like(l)
    gates = w.double() * dw.double()
    g.scatter_(1, ids.long(), gates - w.double() * gates.sum(1, keepdim=True))
    g += st["balance"] * E / n * (p * share - p * (p @ share)[:, None])
    g += st["z"] * 2 / n * lse[:, None] * p
    out = torch.zeros(case["T"], E, dtype=torch.float64, device="cuda")
    out[keep] = g
    return {"loss": torch.stack([st["balance"] * balance + st["z"] * z, balance, z]), "counts": counts.int(),
            "d_logits": out}


def _exact_experts(st, case):
    bits, T, H, I, E, k = (case[n] for n in ("bits", "T", "H", "I", "E", "k"))
    half, cells = 1 << (bits - 1), I * H
    per = 8 // bits

    def matrices(blob):
        codes, steps = blob[:3 * cells // per], blob[3 * cells // per:].clone().view(torch.float16).double()
        # value number v of a byte, then the byte's place in its block
        got = torch.stack([(codes >> (bits * v)) & (2 ** bits - 1) for v in range(per)]).double() - half
        got = got.reshape(per, -1, BLOCK // per).permute(1, 0, 2).reshape(-1, BLOCK) * steps[:, None]
        return got.reshape(3, cells)

    def backward(blob, x, dy):
        wg, wu, wd = matrices(blob)
        g, u = x @ wg.reshape(I, H).t(), x @ wu.reshape(I, H).t()
        q = dy @ wd.reshape(H, I)
        s = torch.sigmoid(g)
        dg, du = q * u * s * (1 + g - g * s), q * g * s
        return dg @ wg.reshape(I, H) + du @ wu.reshape(I, H), torch.sum(q * u * g * s, 1)

    x = st["codes"].double() * torch.exp2(st["scales"].double() - 127).repeat_interleave(BLOCK, 1)
    dy = st["dy"].double()
    dx = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for e in st["live"].tolist():
        t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
        d, v = backward(st["blobs"][e], x[t], dy[t])
        dx[t] += d * st["w"][t, j].double()[:, None]
        dw[t, j] = v
    if st["shared"] is not None:
        dx += backward(st["shared"], x, dy)[0]
    dl = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    w = st["w"].double()
    dl.scatter_(1, st["ids"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))
    return {"dx": dx, "d_logits": dl}
