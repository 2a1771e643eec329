"""GPU checks of the training calls at the edges of what their header allows:
where buffers start, rows that nobody computes, the range of the weights, a
router with a bias, refused steps."""
import numpy as np
import pytest

import workloads as W
from tests import train_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import quantized_expert_ffn_route_b200 as M  # noqa: E402
from tests.test_gpu_train import BF16, F32, MODES, _Case, _dev, _router_case  # noqa: E402


@pytest.fixture(autouse=True)
def _clean_error_word():
    M.moe_device_error(clear=True)
    yield
    torch.cuda.synchronize()
    M.moe_device_error(clear=True)


# ------------------------------------------------------------- workspaces
class _Scratch:
    """n bytes of scratch `off` bytes into a buffer, with guard bytes on both sides."""

    def __init__(self, n, off):
        self.n, self.off = n, off
        self.all = torch.full((off + n + 256,), 255, dtype=torch.uint8, device="cuda")
        assert self.all.data_ptr() % 256 == 0
        self.ws = self.all[off:off + n]

    def check(self):
        torch.cuda.synchronize()
        assert (self.all[:self.off] == 255).all() and (self.all[self.off + self.n:] == 255).all()


@pytest.mark.parametrize("off", [16, 48, 64, 128, 240])
@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_workspace_at_any_16_bytes(mode, off):
    c = _Case(4, 33, 2, 256, 128, 6, True, 41)
    want = c.run(M.MOE_Q8, BF16, F32, mode)
    s = _Scratch(M.moe_expert_ffn_backward_ws_size(4, 33, 2, 256, 128, 6, mode), off)
    got = c.run(M.MOE_Q8, BF16, F32, mode, ws=s.ws)
    s.check()
    assert M.moe_device_error() == 0
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    c.check(*got, F32, mode)


@pytest.mark.parametrize("E", [64, 1200])
def test_balance_and_router_workspace_at_any_16_bytes(E):
    T, H, k, b, z = 700, 256, 3, 0.5, 0.1
    dl, x, w, add = _router_case(T, H, E, BF16, BF16, BF16, 42)
    l = torch.randn(T, E, device="cuda")
    ids = torch.topk(l, k, dim=1)[1].int()
    outs = []
    for off in (0, 16, 240):
        n = M.moe_balance_ws_size(T, E)
        s = _Scratch(n, off)
        cnt, loss = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
        M.moe_balance_loss(l, ids, None, T, E, k, b, z, cnt, loss, s.ws, n)
        s.check()
        n = M.moe_router_backward_ws_size(T, H, E, BF16, BF16, BF16)
        s = _Scratch(n, off)
        dx, dw, db = torch.empty(T, H, device="cuda"), torch.empty_like(w), torch.empty(E, device="cuda")
        M.moe_router_backward(dl, BF16, x, BF16, w, BF16, add, T, H, E, dx, F32, dw, db, s.ws, n)
        s.check()
        outs.append((cnt, loss, dx, dw, db))
    assert M.moe_device_error() == 0
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(outs[0], o))


# ------------------------------------------------- rows that nobody computes
def _with_guards(c, mode, xkind=F32):
    """c.run with guard bytes around its workspace, which starts 16 bytes into a buffer."""
    s = _Scratch(M.moe_expert_ffn_backward_ws_size(c.bits, c.T, c.k, c.H, c.I, c.E, mode), 16)
    out = c.run(xkind, F32, F32, mode, ws=s.ws)
    s.check()
    return out


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T", [1, 2, 3, 33])
def test_expert_backward_one_expert_listed_for_all(T, mode):
    """`active` names one expert over and over, and it has all the rows: while
    the lists hold them, every row is that expert's; where they do not, nothing
    is computed and nothing is added, whatever the workspace held."""
    c = _Case(4, T, 2, 128, 128, 64, True, 43)
    off, act, src, dst = c.perm
    n, e = int(act[0]), int(act[1])
    act = act.clone()
    act[1:1 + n] = e
    off = torch.zeros_like(off)
    off[e + 1:] = 2 * T
    c.perm = (off, act, src, dst)
    dx, dw = _with_guards(c, mode)
    if mode == M.MOE_MODE_GEMM and T == 33:                # 64 times 66 rows
        assert M.moe_device_error() == M.DEVERR_BAD_ROW
        assert (dx == 0).all() and (dw == 0).all()
    else:
        assert M.moe_device_error() == 0
        c.ids[:] = e
        c.check(dx, dw, F32, mode)


BAD_LISTS = ["offsets beyond the rows", "offsets that fall", "expert number too large", "expert number negative",
             "blob off by 8 bytes"]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("T", [1, 3, 33])
@pytest.mark.parametrize("bad", BAD_LISTS)
def test_expert_backward_reports_bad_lists(bad, T, mode):
    """One expert's entry is wrong: it is reported in both forms, its rows add
    nothing and the others are exact."""
    c = _Case(4, T, 2, 128, 128, 6, True, 44)
    off, act, src, dst = (t.clone() for t in c.perm)
    last = int(act[0])
    e = int(act[last])                                     # the last active expert: its end is nobody's start
    table = c.layer.table.clone()
    want = M.DEVERR_BAD_ROW
    if bad == "offsets beyond the rows":
        off[e + 1] = 2 * T + 1
    elif bad == "offsets that fall":
        off[e + 1] = 0
    elif bad == "blob off by 8 bytes":
        table[e] += 8
        want = M.DEVERR_MISALIGNED
    else:
        act[last] = 6 if bad == "expert number too large" else -1
        want = M.DEVERR_BAD_EXPERT
    c.perm = (off, act, src, dst)
    s = _Scratch(M.moe_expert_ffn_backward_ws_size(4, T, 2, 128, 128, 6, mode), 16)
    dx, dw = c.run(F32, F32, F32, mode, table=table, ws=s.ws)
    s.check()
    assert M.moe_device_error() == want
    _, gw = c.check(dx, dw, F32, mode, skip=(e,))
    assert (gw[c.ids == e] == 0).all()


@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_reports_rows_outside_the_permutation(mode):
    T, k = 9, 2
    c = _Case(4, T, k, 128, 128, 6, True, 45)
    off, act, src, dst = (t.clone() for t in c.perm)
    dst[3], dst[10] = T * k, -1
    c.perm = (off, act, src, dst)
    dx, dw = _with_guards(c, mode)
    assert M.moe_device_error() == M.DEVERR_BAD_ROW
    at = [divmod(3, k), divmod(10, k)]
    assert all(float(dw[t, j]) == 0 for t, j in at)
    for t, j in at:
        c.w[t, j] = 0                                      # no share of dx
    rx, rw, ex, ew = R.experts_backward(4, 128, 128, c.blobs, c.shared, c.ids, c.w, c.xv, c.dyv,
                                        0.0 if mode == M.MOE_MODE_GEMV else R.U16)
    assert (np.abs(dx.double().cpu().numpy() - rx) <= ex + R.U32 * np.abs(rx) + 1e-37).all()
    keep = np.ones((T, k), bool)
    for t, j in at:
        keep[t, j] = False
    assert (np.abs(dw.double().cpu().numpy() - rw) <= ew + 1e-37)[keep].all()


# ------------------------------------------------------ range of the weights
def _steps(c, blob):
    """The blob's steps, fp16: gate's and up's, then down's."""
    n = c.H * c.I // 32
    s = blob[3 * c.H * c.I * c.bits // 8:].view(np.float16)
    return s[:2 * n], s[2 * n:]


def _rescale(c, change):
    """Changes every blob's steps in place and lays the experts out again."""
    for blob in list(c.blobs) + ([] if c.shared is None else [c.shared]):
        change(*_steps(c, blob))
    c.layer = M.MoELayer(c.bits, c.H, c.I, c.E, c.k, c.blobs, c.shared)


def _g_noise(c, ua):
    """Expected squares of the norms of dx's and d_topk_w's errors that g's own
    error makes.  g_i sums x_h W_ih, both factors rounded: off by
    2^0.5 ua (sum_h (x_h W_ih)^2)^0.5, independently for each i.  To first order
    dg_i is off by q u F' of that, F = s + a (1 - s), F' = s (1 - s) (2 + g (1 - 2 s)),
    du_i by q F and <q, a u> by q u F; dx sums them over rows of Wg and Wu.  At
    |g| about 1 this is one of the ten roundings below; it grows with |g|."""
    ex2, ew2 = 0.0, 0.0
    for e in range(c.E + (c.shared is not None)):
        Wg, Wu, Wd = R.matrices(c.bits, c.H, c.I, c.blobs[e] if e < c.E else c.shared)
        t, j = np.nonzero(c.ids == e) if e < c.E else (np.arange(c.T), None)
        x, w = c.xv[t], (c.w[t, j].astype(np.float64) if e < c.E else np.ones(c.T))[:, None]
        g, u, q = x @ Wg.T, x @ Wu.T, c.dyv[t] @ Wd
        s = 1 / (1 + np.exp(-g))
        F, dF = s + g * s * (1 - s), s * (1 - s) * (2 + g * (1 - 2 * s))
        var = 2 * ua * ua * ((x * x) @ (Wg * Wg).T)
        size = np.abs(q * u * dF) * np.linalg.norm(Wg, axis=1) + np.abs(q * F) * np.linalg.norm(Wu, axis=1)
        ex2 += (w * w * size * size * var).sum()
        ew2 += (q * u * F * q * u * F * var).sum() if e < c.E else 0.0
    return ex2, ew2


def _check_weights(c, dx, dw, mode):
    """c.check with one more term.  The gradients of g and u are stored in fp16
    times a power of two 2^15 / B' with B' at most 4 times their bound
    B = half^2 max|step of gate, up| max|step of down| |x|_1 |dy|_1 (the weights'
    part and the rows', each taken up to a power of two).  fp16's smallest step
    is 2^-24: a stored value is off by up to 2^-25 2^-15 4 B = 2^-38 B."""
    gemm = mode == M.MOE_MODE_GEMM
    rx, rw, ex, ew = R.experts_backward(c.bits, c.H, c.I, c.blobs, c.shared, c.ids, c.w, c.xv, c.dyv,
                                        R.U16 if gemm else 0.0)
    lost = 0.0                                             # the same for dx's norm, each i apart
    if gemm:
        l1 = np.abs(c.xv).sum(1) * np.abs(c.dyv).sum(1)
        for e in range(c.E + (c.shared is not None)):
            blob = c.blobs[e] if e < c.E else c.shared
            gu, d = (float(np.abs(s.astype(np.float64)).max()) for s in _steps(c, blob))
            floor = 2.0 ** -38 * 4.0 ** (c.bits - 1) * gu * d * l1
            Wg, Wu, _ = R.matrices(c.bits, c.H, c.I, blob)
            col = np.abs(Wg).sum(0) + np.abs(Wu).sum(0)
            wt = np.where(c.ids == e, c.w, 0).sum(1) if e < c.E else 1.0
            ex = ex + 1.1 * (wt * floor)[:, None] * col
            lost += ((wt * floor) ** 2).sum() * ((Wg * Wg).sum() + (Wu * Wu).sum())
    gx, gw = dx.double().cpu().numpy(), dw.double().cpu().numpy()
    assert np.isfinite(gx).all() and np.isfinite(gw).all()
    assert (np.abs(gx - rx) <= ex + 1e-37).all(), (np.abs(gx - rx) / (ex + 1e-37)).max()
    assert (np.abs(gw - rw) <= ew + 1e-37).all(), (np.abs(gw - rw) / (ew + 1e-37)).max()
    # as in c.check: about ten independent roundings of half a step along a value's path; and g's, and the
    # smallest steps
    half = R.U16 if gemm else 32 * R.U32
    for err, size, g2, l2 in zip((gx - rx, gw - rw), (rx, rw), _g_noise(c, half), (lost, 0.0)):
        assert (err ** 2).sum() <= 10 * half ** 2 * (size ** 2).sum() + g2 + l2


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("gu,down", [(-9, -9), (-9, 9), (6, 6), (12, 16), (16, -9)])
@pytest.mark.parametrize("bits,T,E", [(4, 20, 6), (2, 20, 6), (4, 300, 2)])
def test_expert_backward_weight_scales_do_not_matter(bits, T, E, gu, down, mode):
    """Steps from about 2^-15 to 2^10, gate and up apart from down: the inner
    gradients keep their bits and stay finite.  x undoes gate's scale, so that
    g keeps its size."""
    c = _Case(bits, T, 2, 256, 128, E, True, 46)

    def change(s, d):
        s[:], d[:] = np.ldexp(s, gu), np.ldexp(d, down)
        assert np.isfinite(s).all() and np.isfinite(d).all()
    _rescale(c, change)
    c.x *= np.float32(2.0 ** -gu)
    dx, dw = c.run(F32, F32, F32, mode)
    assert M.moe_device_error() == 0
    _check_weights(c, dx, dw, mode)


@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_one_large_block_of_weights(mode):
    """A block of 32 weights 2^8 times the others, in up and in down."""
    c = _Case(4, 40, 2, 256, 128, 6, True, 47)

    def change(s, d):
        s[c.H * c.I // 32 + 77] *= 256
        d[99] *= 256
    _rescale(c, change)
    dx, dw = c.run(M.MOE_Q8, F32, F32, mode)
    assert M.moe_device_error() == 0
    _check_weights(c, dx, dw, mode)


@pytest.mark.parametrize("bits", [2, 4])
def test_expert_backward_reports_weights_beyond_fp16(bits):
    """A step whose lowest code's weight is outside fp16: exact on CUDA cores,
    reported by the tensor cores' form, which keeps it to its expert."""
    c = _Case(bits, 20, 2, 128, 128, 6, False, 48)
    c.x *= np.float32(1e-6)
    top = np.float16(65504 / 2 ** (bits - 1))              # the largest that is inside
    for step, bad in ((top, False), (np.nextafter(top, np.float16(np.inf)), True)):
        s, _ = _steps(c, c.blobs[3])
        s[5] = -step
        c.layer = M.MoELayer(bits, 128, 128, 6, 2, c.blobs, None)
        dx, dw = c.run(F32, F32, F32, M.MOE_MODE_GEMV)
        assert M.moe_device_error() == 0
        _check_weights(c, dx, dw, M.MOE_MODE_GEMV)
        dx, dw = c.run(F32, F32, F32, M.MOE_MODE_GEMM)
        assert M.moe_device_error() == (M.DEVERR_NONFINITE if bad else 0)
        others = _dev((c.ids != 3).all(1))
        assert torch.isfinite(dx[others]).all() and torch.isfinite(dw[_dev(c.ids != 3)]).all()


@pytest.mark.parametrize("side", ["up", "down"])
def test_expert_backward_largest_steps_at_the_end(side):
    """Matrices whose steps take a block several rounds to look through, the
    large ones (2^14 times the others) in the last rows: missed, they would
    take the inner gradients past fp16's end."""
    c = _Case(4, 6, 1, 4096, 1536, 2, False, 50, sigma=0.02)

    def change(s, d):
        t = s if side == "up" else d
        n = c.H * c.I // 32 // 16
        t[-n:] = np.ldexp(t[-n:], 14)
        assert np.isfinite(t).all()
    _rescale(c, change)
    dx, dw = c.run(M.MOE_Q8, BF16, F32, M.MOE_MODE_GEMM)
    assert M.moe_device_error() == 0
    _check_weights(c, dx, dw, M.MOE_MODE_GEMM)


@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_one_large_value_a_token(mode):
    """Each token's x and dy have one value 2^10 times the others."""
    c = _Case(4, 40, 2, 2048, 128, 6, True, 49, sigma=0.02)
    c.x[:, 5] *= 1024
    c.dy[:, 1900] *= 1024
    dx, dw = c.run(F32, F32, F32, mode)
    assert M.moe_device_error() == 0
    _check_weights(c, dx, dw, mode)


# ----------------------------------------------------------------- TrainStep
@pytest.mark.parametrize("wdt,E,T", [("bf16", 22, 37), ("f32", 22, 37), ("bf16", 24, 37), ("bf16", 13, 3)])
def test_train_step_with_a_router_bias(wdt, E, T):
    """A router with a bias, E a multiple of 8 and not: logits, losses and every
    gradient against the 64-bit chain on the same routing and checkpoint."""
    H, I, k = 256, 128, 3
    rng = np.random.default_rng(E + T)
    bias = rng.standard_normal(E).astype(np.float32)
    lay = W.make_layer(9, 4, H, I, E, k, shared=True, w_dtype=wdt, bias=bias)
    g = M.MoELayer(4, H, I, E, k, lay.blobs, lay.shared, lay.w_router, wdt, bias)
    x = W.bf16_bits_to_f32(W.make_tokens(8, T, H, "bf16")).astype(np.float32)
    dy = rng.standard_normal((T, H)).astype(np.float32)
    mask = np.arange(T) % 3 != 1
    dy[~mask] = 0
    b, z, dl = 0.5, 0.01, -1.5
    step = M.TrainStep(g, T, BF16, dy_dtype=F32, dx_dtype=F32, balance_coef=b, z_coef=z)
    _, loss = step.forward(_dev(x).bfloat16(), token_mask=_dev(mask))
    out = step.backward(_dev(dy), d_loss=torch.tensor([dl], device="cuda"))
    torch.cuda.synchronize()
    assert M.moe_device_error() == 0
    wr = (W.bf16_bits_to_f32(lay.w_router) if wdt == "bf16" else lay.w_router).astype(np.float64)
    logits = step.bufs.logits[:T * E].cpu().numpy().reshape(T, E)
    # a sum of H products and the bias in fp32, a tensor core cutting instead of rounding
    size = np.abs(x.astype(np.float64)) @ np.abs(wr).T + np.abs(bias)
    assert (np.abs(logits - (x.astype(np.float64) @ wr.T + bias)) <= 2 * (H + 4) * R.U32 * size).all()
    ids = step.bufs.ids[:T * k].cpu().numpy().reshape(T, k)
    w = step.bufs.w[:T * k].cpu().numpy().reshape(T, k)
    counts, losses, lgrad = R.balance(logits, ids, mask, E, b, z)
    assert np.array_equal(step.counts.cpu().numpy(), counts)
    # each term is a mean of positive numbers: sums of E or T fp32 terms, exponentials of differences up to
    # `spread`; the square's factor twice its own, lse below max|l| + log E
    per = (R.spread(logits, mask) + E + T + 24) * R.U32
    lim = 4 * per * np.array([b * losses[1] + z * losses[2] + z, losses[1], losses[2] + 1])
    assert (np.abs(loss.double().cpu().numpy() - losses)[:3] <= lim).all() and loss[3] == losses[3]
    xv = R.act8(x)[2]
    dx, dw, ex, ew = R.experts_backward(4, H, I, lay.blobs, lay.shared, ids, w, xv, dy.astype(np.float64),
                                        R.U16 if T > 4 else 0.0)
    want = dl * lgrad + R.gates(ids, w, dw, E, mask)
    # d_logits: the gates' error through dw, fp32 noise of both terms, the rounding to its type
    bound = np.zeros((T, E))
    for t in np.nonzero(mask)[0]:
        np.add.at(bound[t], ids[t], w[t] * (ew[t] + (w[t] * ew[t]).sum()) +
                  (k + 8) * R.U32 * w[t] * (np.abs(dw[t]) + np.abs(w[t] * dw[t]).sum()))
    N = mask.sum()
    f = counts[:E] / (N * k)
    p = np.exp(logits.astype(np.float64) - logits.max(1, keepdims=True))
    p = np.where(mask[:, None], p / p.sum(1, keepdims=True), 0)
    top = np.abs(logits).max() + np.log(E)
    bound += abs(dl) * p * (b * E / N * (f + (f * p).sum(1, keepdims=True)) + z * 2 / N * top) * 2 * per
    half = R.UBF if wdt == "bf16" else R.U32
    gdl = step.d_logits.double().cpu().numpy()
    assert (np.abs(gdl - want) <= bound + half * 1.01 * np.abs(want) + 1e-37).all()
    assert (gdl[~mask] == 0).all()
    # the router's products of the d_logits it was given: fp32 sums, cut or rounded, and the result's rounding
    def close(got, want, size, terms, half):
        lim = 2 * (terms + 4) * R.U32 * size
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= lim + half * 1.01 * (np.abs(want) + lim) + 1e-37).all(), (err / (lim + 1e-37)).max()
    close(out["d_w_router"], gdl.T @ xv, np.abs(gdl).T @ np.abs(xv), T, half)
    close(out["d_bias"], gdl.sum(0), np.abs(gdl).sum(0), T, R.U32)
    got = out["dx"].double().cpu().numpy()
    lim = 2 * (E + 4) * R.U32 * (np.abs(gdl) @ np.abs(wr) + np.abs(dx) + ex)
    assert (np.abs(got - (dx + gdl @ wr)) <= ex + lim + 1e-37).all()


def test_train_step_refuses_before_it_launches_and_recovers():
    """A refused forward() leaves the layer's buffers as they were and no
    backward(); the next whole forward() has one again."""
    H, I, E, k, T = 256, 128, 16, 2, 8
    lay = W.make_layer(5, 4, H, I, E, k, shared=False, w_dtype="bf16")
    g = M.MoELayer(4, H, I, E, k, lay.blobs, None, lay.w_router, "bf16")
    step = M.TrainStep(g, T, BF16)
    x, dy = torch.randn(T, H, device="cuda").bfloat16(), torch.randn(T, H, device="cuda")
    step.forward(x)
    want = [v.clone() for v in step.backward(dy).values()]
    logits = step.bufs.logits.clone()
    launches = M.moe_kernel_launches()
    for bad in (x[:T - 1], x.float(), x.cpu(), x.t().contiguous().t(), x.float().cpu().numpy()):
        with pytest.raises((ValueError, TypeError)):
            step.forward(bad)
        with pytest.raises(RuntimeError, match="forward"):
            step.backward(dy)
    with pytest.raises(ValueError):
        step.forward(x, token_mask=torch.ones(T - 1, dtype=torch.bool, device="cuda"))
    assert M.moe_kernel_launches() == launches
    step.forward(x)
    with pytest.raises(ValueError):
        step.backward(dy.bfloat16())
    with pytest.raises(ValueError):
        step.backward(dy, d_loss=torch.ones(1))
    assert torch.equal(step.bufs.logits, logits)
    assert all(torch.equal(a, b) for a, b in zip(step.backward(dy).values(), want))
    assert M.moe_device_error() == 0
