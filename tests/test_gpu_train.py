"""GPU checks of the training calls against plain 64-bit definitions
(tests/train_ref.py), at the sizes and masks where they can go wrong."""
import numpy as np
import pytest

import workloads as W
from tests import train_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import quantized_expert_ffn_route_b200 as M  # noqa: E402

F32, BF16 = M.MOE_F32, M.MOE_BF16


@pytest.fixture(autouse=True)
def _clean_error_word():
    M.moe_device_error(clear=True)
    yield
    torch.cuda.synchronize()
    M.moe_device_error(clear=True)


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def _tt(code):
    return torch.bfloat16 if code == BF16 else torch.float32


def _half(code):
    return R.UBF if code == BF16 else R.U32


def _guarded(n, dtype, fill):
    """A buffer of n values with 64 more of `fill` behind them."""
    t = torch.full((n + 64,), fill, dtype=dtype, device="cuda")
    return t


# ------------------------------------------------------ 8-bit checkpoints
def _act_case(kind, T, H, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, H)) * np.exp(2 * rng.standard_normal((T, 1)))).astype(np.float32)
    if kind == "special":
        b = x.reshape(-1, 32)
        n = b.shape[0]
        b[0 % n] = 0.0
        b[1 % n, 3] = np.nan
        b[2 % n, 31] = np.inf
        b[3 % n, 0] = -np.inf
        b[4 % n] = 1e-42                                   # below the smallest normal number
        b[5 % n] = np.float32(3.3895e38) * np.sign(b[5 % n])  # the largest of bf16
        b[6 % n] = 2.0 ** -126
        b[7 % n, :2] = [127.5, -127.4]
        b[8 % n, :] = np.arange(32) + 0.5                  # ties
        b[9 % n, :] = np.linspace(-1, 1, 32) * np.float32(2.0 ** -121 * 1.9999)
        b[10 % n, 5] = np.finfo(np.float32).max
        b[11 % n, :] = -0.0
    return x


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H", [(1, 32), (1, 2048), (3, 96), (77, 1184), (300, 512)])
@pytest.mark.parametrize("kind", ["normal", "special"])
def test_act8_is_exact(dtype, T, H, kind):
    x = _dev(_act_case(kind, T, H, T + H)).to(_tt(dtype))
    q, s, v = R.act8(x.float().cpu().numpy())
    codes, scales = _guarded(T * H, torch.int8, 77), _guarded(T * H // 32, torch.uint8, 99)
    y = _guarded(T * H, _tt(dtype), 5.0)
    M.moe_act_pack8(x, dtype, T, H, codes, scales)
    M.moe_act_unpack8(codes, scales, T, H, y, dtype)
    torch.cuda.synchronize()
    assert np.array_equal(codes[:T * H].cpu().numpy().reshape(T, H), q)
    assert np.array_equal(scales[:T * H // 32].cpu().numpy().reshape(T, -1), s)
    got = y[:T * H].double().cpu().numpy().reshape(T, H)
    assert np.array_equal(got, v, equal_nan=True)
    assert (codes[T * H:] == 77).all() and (scales[T * H // 32:] == 99).all() and (y[T * H:] == 5.0).all()


def test_act8_unpacks_to_the_other_type_exactly():
    x = _dev(_act_case("normal", 9, 256, 3))
    codes = torch.empty(9, 256, dtype=torch.int8, device="cuda")
    scales = torch.empty(9, 8, dtype=torch.uint8, device="cuda")
    a, b = torch.empty(9, 256, device="cuda"), torch.empty(9, 256, dtype=torch.bfloat16, device="cuda")
    M.moe_act_pack8(x, F32, 9, 256, codes, scales)
    M.moe_act_unpack8(codes, scales, 9, 256, a, F32)
    M.moe_act_unpack8(codes, scales, 9, 256, b, BF16)
    assert torch.equal(a, b.float())


# ----------------------------------------------------------- balance loss
def _route_case(T, E, k, seed, mask):
    rng = np.random.default_rng(seed)
    l = (2 * rng.standard_normal((T, E)) + rng.standard_normal(E)).astype(np.float32)
    if mask == "inf":                                      # experts shut off, and one row with nothing left
        l[:, rng.permutation(E)[:max(0, E - k - 1)]] = -np.inf
        l[T // 2] = -np.inf
        l[0, 0] = np.finfo(np.float32).min
    ids = np.argsort(-l, 1, kind="stable")[:, :k].astype(np.int32)
    keep = None
    if mask == "some":
        keep = (rng.random(T) < 0.6).astype(np.uint8)
    elif mask == "none left":
        keep = np.zeros(T, np.uint8)
    elif mask == "nan outside":
        keep = np.ones(T, np.uint8)
        keep[::3] = 0
        l[::3] = np.nan
        ids[::3] = -5
    s = np.exp(np.take_along_axis(np.where(np.isfinite(l), l, 0), np.clip(ids, 0, E - 1), 1).astype(np.float64) * 0.3)
    w = (s / s.sum(1, keepdims=True)).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    if mask == "nan outside":
        w[::3] = dw[::3] = np.nan
    return l, ids, w, dw, keep


BALANCE = [(1, 1, 1), (1, 16, 2), (8, 16, 2), (33, 130, 3), (65, 512, 10), (40, 1000, 32), (9, 1021, 7), (5, 1025, 1),
           (12, 1028, 4), (4, 24576, 10), (3, 32767, 32), (700, 64, 4)]


@pytest.mark.parametrize("T,E,k", BALANCE)
@pytest.mark.parametrize("mask", ["all", "some", "none left", "nan outside", "inf"])
def test_balance_loss_and_gradient(T, E, k, mask):
    if mask == "inf" and E < 8:
        pytest.skip("no expert to shut off")
    l, ids, w, dw, keep = _route_case(T, E, k, T * 31 + E, mask)
    on = np.ones(T, bool) if keep is None else keep != 0
    b, z, g = 0.8, 0.05, -1.7
    counts, losses, grad = R.balance(np.where(on[:, None], l, 0), np.where(on[:, None], ids, 0), keep, E, b, z)
    ld, idd, wd, dwd = _dev(l), _dev(ids), _dev(w), _dev(dw)
    md = None if keep is None else _dev(keep)
    cd, loss = _guarded(E + 1, torch.int32, 123), _guarded(4, torch.float32, 9.0)
    n = M.moe_balance_ws_size(T, E)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    M.moe_balance_loss(ld, idd, md, T, E, k, b, z, cd, loss, ws, n)
    assert M.moe_device_error() == 0
    assert np.array_equal(cd[:E + 1].cpu().numpy(), counts)
    assert (cd[E + 1:] == 123).all() and (loss[4:] == 9.0).all()
    # relative error of one p: the difference l - max is rounded once (its error
    # grows with its size), exp and the division add a few steps, the sum of E
    # terms at most one step an addition along a lane's chain and the joins
    per = (R.spread(l, on) + E / 32 + 24) * R.U32
    got = loss[:4].cpu().numpy().astype(np.float64)
    assert got[3] == losses[3]
    # sums over rows: one step an addition of a warp's rows, then 64 bits
    # (every row adds a non-negative share); lse is off by `per` steps of its own or of 1
    zs = 2 * (losses[2] + np.sqrt(losses[2]))
    size = [b * losses[1] + z * zs, losses[1], zs]
    for i in range(3):
        # a row of the type's lowest value alone has lse = -3.4e38; its square is outside fp32: inf
        if abs(losses[i]) > np.finfo(np.float32).max:
            assert got[i] == np.inf
        else:
            assert abs(got[i] - losses[i]) <= (2 * per + (T / 8 + 8) * R.U32) * size[i] + 1e-30
    # the row's lse against cancellation: |lse| <= max|l| + log E enters with its own rounding
    top = np.abs(np.where(np.isfinite(l) & on[:, None], l, 0)).max() + np.log(E) if on.any() else 0
    N = max(1, on.sum())
    f = counts[:E] / (N * k)
    for dtype in (F32, BF16):
        for gate in (False, True):
            want = g * grad
            p = np.zeros_like(grad)
            for t in np.nonzero(on)[0]:
                m = l[t].max()
                if m > -np.inf:
                    e = np.exp(l[t].astype(np.float64) - m)
                    p[t] = e / e.sum()
            bound = abs(g) * p * (b * E / N * (f + (f * p).sum(1, keepdims=True)) + z * 2 / N * top) * 2 * per
            if gate:
                want = want + R.gates(np.where(on[:, None], ids, 0), np.where(on[:, None], w, 0),
                                      np.where(on[:, None], dw, 0), E, on)
                wdw = np.where(on[:, None], np.abs(w) * (np.abs(dw) + np.abs(w * dw).sum(1, keepdims=True)), 0)
                for t in np.nonzero(on)[0]:
                    np.add.at(bound[t], ids[t], wdw[t] * (k + 8) * R.U32)
            bound = bound + _half(dtype) * 1.01 * np.abs(want) + 1e-37
            dl = _guarded(T * E, _tt(dtype), 3.0)
            M.moe_route_backward(ld, idd if gate else None, wd if gate else None, dwd if gate else None, md, cd,
                                 torch.tensor([g], device="cuda"), T, E, k, b, z, dl, dtype)
            out = dl[:T * E].double().cpu().numpy().reshape(T, E)
            assert (np.abs(out - want) <= bound).all(), (dtype, gate, (np.abs(out - want) / bound).max())
            assert (out[~on] == 0).all() and (dl[T * E:] == 3.0).all()
    assert M.moe_device_error() == 0


@pytest.mark.parametrize("E", [40, 2000])
def test_route_backward_gates_only_and_repeated_ids(E):
    T, k = 6, 5
    rng = np.random.default_rng(E)
    ids = rng.integers(0, 3, (T, k)).astype(np.int32)      # the same expert several times in a row
    w, dw = rng.random((T, k)).astype(np.float32), rng.standard_normal((T, k)).astype(np.float32)
    outs = []
    for _ in range(2):
        dl = torch.full((T, E), 7.0, device="cuda")
        M.moe_route_backward(None, _dev(ids), _dev(w), _dev(dw), None, None, None, T, E, k, 1.0, 1.0, dl, F32)
        outs.append(dl)
    want = R.gates(ids, w, dw, E)
    # k products and additions of each sum, a step each
    size = np.zeros_like(want)
    for t in range(T):
        np.add.at(size[t], ids[t], np.abs(w[t]) * (np.abs(dw[t]) + np.abs(w[t] * dw[t]).sum()))
    assert (np.abs(outs[0].double().cpu().numpy() - want) <= (2 * k + 8) * R.U32 * size + 1e-37).all()
    assert torch.equal(outs[0], outs[1])


def test_balance_reports_bad_ids_and_logits():
    T, E, k = 4, 16, 2
    l = np.zeros((T, E), np.float32)
    ids = np.tile(np.array([0, 1], np.int32), (T, 1))
    n = M.moe_balance_ws_size(T, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    cd, loss = torch.empty(E + 1, dtype=torch.int32, device="cuda"), torch.empty(4, device="cuda")
    ids[1, 1], ids[2, 0] = 16, -1
    M.moe_balance_loss(_dev(l), _dev(ids), None, T, E, k, 1.0, 1.0, cd, loss, ws, n)
    assert M.moe_device_error() == M.DEVERR_BAD_EXPERT
    assert cd[0] == 3 and cd[1] == 3 and cd[:E].sum() == 6 and cd[E] == T
    dl = torch.empty(T, E, device="cuda")
    one = torch.ones(T, k, device="cuda")
    M.moe_route_backward(None, _dev(ids), one, one, None, None, None, T, E, k, 0.0, 0.0, dl, F32)
    assert M.moe_device_error() == M.DEVERR_BAD_EXPERT
    ids[:] = [0, 1]
    for bad in (np.nan, np.inf):
        l2 = l.copy()
        l2[2, 5] = bad
        M.moe_balance_loss(_dev(l2), _dev(ids), None, T, E, k, 1.0, 1.0, cd, loss, ws, n)
        assert M.moe_device_error() == M.DEVERR_NONFINITE and torch.isnan(loss[:3]).all()
        M.moe_route_backward(_dev(l2), None, None, None, None, cd, None, T, E, k, 1.0, 1.0, dl, F32)
        assert M.moe_device_error() == M.DEVERR_NONFINITE
        assert torch.isnan(dl[2]).all() and torch.isfinite(dl[[0, 1, 3]]).all()


def test_balance_of_no_tokens():
    cd, loss = torch.full((17,), 4, dtype=torch.int32, device="cuda"), torch.full((4,), 4.0, device="cuda")
    M.moe_balance_loss(None, None, None, 0, 16, 2, 1.0, 1.0, cd, loss)
    assert (cd == 0).all() and (loss == 0).all()


# ---------------------------------------------------------------- experts
def _perm(ids, E):
    T, k = ids.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    n = M.moe_permute_ws_size(T, k, E)
    off, act = torch.empty(E + 1, **i32), torch.empty(1 + min(E, T * k), **i32)
    src, dst = torch.empty(T * k, **i32), torch.empty(T * k, **i32)
    M.moe_permute(_dev(ids), T, k, E, off, src, dst, act, torch.empty(max(16, n), dtype=torch.uint8, device="cuda"), n)
    return off, act, src, dst


class _Case:
    def __init__(self, bits, T, k, H, I, E, shared, seed, skew=False, sigma=0.05):
        rng = np.random.default_rng(seed)
        g = np.random.Generator(np.random.PCG64(seed))
        self.bits, self.T, self.k, self.H, self.I, self.E = bits, T, k, H, I, E
        # 11-bit steps: a weight is then no exact fp16 number
        self.blobs = np.stack([W.random_expert_blob(g, bits, H, I, sigma, 11) for _ in range(E)])
        self.shared = W.random_expert_blob(g, bits, H, I, sigma, 11) if shared else None
        if skew:                                           # most tokens to two experts, several experts without any
            self.ids = np.stack([np.concatenate([[0], 1 + rng.permutation(max(1, (E - 1) // 2))])[:k]
                                 for _ in range(T)]).astype(np.int32)
        else:
            self.ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
        w = rng.random((T, k)) + 0.05
        self.w = (w / w.sum(1, keepdims=True)).astype(np.float32)
        self.x = (rng.standard_normal((T, H)) * np.exp(rng.standard_normal((T, 1)))).astype(np.float32)
        self.dy = (rng.standard_normal((T, H)) * np.exp(3 * rng.standard_normal((T, 1))) * 1e-4).astype(np.float32)
        self.layer = M.MoELayer(bits, H, I, E, k, self.blobs, self.shared)
        self.perm = _perm(self.ids, E)

    def run(self, xkind, dyd, dxd, mode, active=None, table=None, ws=None):
        T, k, H = self.T, self.k, self.H
        if xkind == M.MOE_Q8:
            x = torch.empty(T, H, dtype=torch.int8, device="cuda")
            xs = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
            M.moe_act_pack8(_dev(self.x), F32, T, H, x, xs)
            self.xv = R.act8(self.x)[2]
        else:
            x, xs = _dev(self.x).to(_tt(xkind)), None
            self.xv = x.double().cpu().numpy()
        dy = _dev(self.dy).to(_tt(dyd))
        self.dyv = dy.double().cpu().numpy()
        dx, dw = _guarded(T * H, _tt(dxd), 8.0), _guarded(T * k, torch.float32, 8.0)
        n = M.moe_expert_ffn_backward_ws_size(self.bits, T, k, H, self.I, self.E, mode)
        # scratch needs no contents: NaN patterns must not come through
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda") if ws is None else ws
        off, act, src, dst = self.perm
        M.moe_expert_ffn_backward(self.bits, self.layer.table if table is None else table, off,
                                  act if active is None else active, src, dst, _dev(self.w), x, xkind, xs, dy, dyd, T, k,
                                  H, self.I, self.E, self.layer.shared, dx, dxd, dw, mode, ws, n)
        torch.cuda.synchronize()
        assert (dx[T * H:] == 8.0).all() and (dw[T * k:] == 8.0).all()
        return dx[:T * H].view(T, H), dw[:T * k].view(T, k)

    def check(self, dx, dw, dxd, mode, skip=()):
        ua = 0.0 if mode == M.MOE_MODE_GEMV else R.U16
        rx, rw, ex, ew = R.experts_backward(self.bits, self.H, self.I, self.blobs, self.shared, self.ids, self.w,
                                            self.xv, self.dyv, ua, R.U32, skip)
        gx, gw = dx.double().cpu().numpy(), dw.double().cpu().numpy()
        ex = ex + _half(dxd) * (np.abs(rx) + ex) * 1.01
        assert (np.abs(gx - rx) <= ex + 1e-37).all(), (np.abs(gx - rx) / (ex + 1e-37)).max()
        assert (np.abs(gw - rw) <= ew + 1e-37).all(), (np.abs(gw - rw) / (ew + 1e-37)).max()
        # roundings are independent: about ten of half a step each along a value's path, in quadrature
        rms = np.sqrt(10.0) * (ua or 32 * R.U32) + _half(dxd)
        assert np.linalg.norm(gx - rx) <= rms * np.linalg.norm(rx) + 1e-37
        return gx, gw


SHAPES = [  # bits, T, k, H, I, E, shared, skew
    (4, 1, 1, 128, 128, 1, False, False),
    (4, 1, 2, 256, 128, 16, True, False),
    (2, 1, 3, 384, 256, 5, True, False),
    (4, 7, 2, 256, 384, 4, False, False),
    (2, 17, 4, 640, 128, 9, True, False),
    (4, 65, 3, 256, 256, 11, True, True),
    (2, 300, 2, 256, 128, 3, False, True),
    (4, 700, 1, 128, 128, 2, True, False),
]
MODES = [M.MOE_MODE_GEMV, M.MOE_MODE_GEMM]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bits,T,k,H,I,E,shared,skew", SHAPES)
def test_expert_backward(bits, T, k, H, I, E, shared, skew, mode):
    c = _Case(bits, T, k, H, I, E, shared, 100 + T + H, skew)
    kinds = [(M.MOE_Q8, BF16, BF16), (F32, F32, F32)] + ([(BF16, F32, BF16)] if T < 100 else [])
    for xkind, dyd, dxd in kinds:
        dx, dw = c.run(xkind, dyd, dxd, mode)
        assert M.moe_device_error() == 0
        c.check(dx, dw, dxd, mode)
        dx2, dw2 = c.run(xkind, dyd, dxd, mode)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2)        # no order of scheduling in the results


@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_large_shapes(mode):
    """The widest hidden and intermediate sizes."""
    c = _Case(2, 3, 2, 8192, 128, 3, False, 9)
    dx, dw = c.run(BF16, BF16, F32, mode)
    c.check(dx, dw, F32, mode)
    c = _Case(4, 3, 1, 128, 4096, 2, True, 10)
    dx, dw = c.run(BF16, F32, BF16, mode)
    c.check(dx, dw, BF16, mode)
    assert M.moe_device_error() == 0


@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_scales_do_not_matter(mode):
    """Tiny and huge gradients and activations: the result scales with them."""
    c = _Case(4, 40, 2, 256, 128, 6, True, 21)
    base = c.dy.copy()
    for scale in (1e-30, 1.0, 1e25):
        c.dy = (base * np.float32(scale)).astype(np.float32)
        dx, dw = c.run(F32, F32, F32, mode)
        c.check(dx, dw, F32, mode)
    c.dy = base
    c.dy[3] = 0.0                                          # a token without a gradient, and one without an input
    c.x[5] = 0.0
    dx, dw = c.run(F32, F32, F32, mode)
    c.check(dx, dw, F32, mode)
    assert (dx[3] == 0).all() and (dw[3] == 0).all() and (dw[5] == 0).all()


@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_keeps_nan_to_its_token(mode):
    c = _Case(4, 20, 2, 256, 128, 4, True, 22)
    c.dy[7, 100] = np.nan
    c.x[9, 3] = np.inf
    for kind in (F32, M.MOE_Q8):
        dx, dw = c.run(kind, F32, F32, mode)
        ok = np.ones(20, bool)
        ok[[7, 9]] = False
        assert torch.isfinite(dx[_dev(ok)]).all() and torch.isfinite(dw[_dev(ok)]).all()
        assert torch.isnan(dx[7]).all() and torch.isnan(dw[7]).all() and not torch.isfinite(dx[9]).any()


@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_of_missing_experts(mode):
    """An expert without a blob, and one left out of `active`, add nothing."""
    c = _Case(4, 30, 3, 256, 128, 6, True, 23)
    table = c.layer.table.clone()
    table[2] = 0
    dx, dw = c.run(F32, F32, F32, mode, table=table)
    assert M.moe_device_error() == M.DEVERR_NULL_BLOB
    gx, gw = c.check(dx, dw, F32, mode, skip=(2,))
    assert (gw[c.ids == 2] == 0).all()
    act = c.perm[1].cpu().numpy()
    rest = [e for e in act[1:1 + act[0]] if e != 4]
    less = np.zeros_like(act)
    less[0], less[1:1 + len(rest)] = len(rest), rest
    dx, dw = c.run(F32, F32, F32, mode, active=_dev(less))
    assert M.moe_device_error() == 0
    gx, gw = c.check(dx, dw, F32, mode, skip=(4,))
    assert (gw[c.ids == 4] == 0).all()


def test_expert_backward_auto_mode_and_other_stream():
    c = _Case(4, 20, 2, 256, 128, 4, True, 24)
    want = c.run(F32, F32, F32, M.MOE_MODE_AUTO)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = c.run(F32, F32, F32, M.MOE_MODE_AUTO)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("mode", MODES)
def test_expert_backward_many_experts(mode):
    """More experts than one block lists at a time, most of them without tokens."""
    c = _Case(2, 150, 4, 128, 128, 700, True, 25)
    dx, dw = c.run(BF16, BF16, BF16, mode)
    assert M.moe_device_error() == 0
    c.check(dx, dw, BF16, mode)


@pytest.mark.parametrize("T", [0, 2, 33])
def test_expert_backward_inconsistent_lists_stay_in_bounds(T):
    """An `active` list that names an expert many times over, or offsets that
    overlap: nothing is written outside the buffers, and it is reported."""
    T = max(T, 20)
    c = _Case(4, T, 2, 128, 128, 64, True, 26)
    off, act, src, dst = c.perm
    n = int(act[0])
    twice = act.clone()
    twice[1:1 + n] = act[1]
    wide = off.clone()
    wide[:64] = 0
    wide[1:] = T * 2
    for mode in MODES:
        c.perm = (wide, twice, src, dst)
        c.run(F32, F32, F32, mode)                         # checks its guard values
        bits = M.moe_device_error()
        if mode == M.MOE_MODE_GEMM:
            assert bits == M.DEVERR_BAD_ROW
    c.perm = (off, act, src, dst)
    dx, dw = c.run(F32, F32, F32, M.MOE_MODE_GEMM)
    c.check(dx, dw, F32, M.MOE_MODE_GEMM)


def test_expert_backward_offsets_beyond_32_bits():
    """Rows x hidden above 2^31: sampled tokens against the definition."""
    T, k, H, I, E = (1 << 17) + 9, 8, 2048, 128, 8
    assert T * (k + 1) * H > 1 << 31
    g = np.random.Generator(np.random.PCG64(27))
    blobs = np.stack([W.random_expert_blob(g, 4, H, I, 0.02) for _ in range(E)])
    layer = M.MoELayer(4, H, I, E, k, blobs, blobs[0])
    torch.manual_seed(27)
    x = torch.randn(T, H, device="cuda").bfloat16()
    dy = torch.randn(T, H, device="cuda").bfloat16()
    ids = torch.argsort(torch.rand(T, E, device="cuda"), 1).int().contiguous()
    w = torch.softmax(torch.randn(T, k, device="cuda"), 1)
    off, act, src, dst = _perm(ids.cpu().numpy(), E)
    n = M.moe_expert_ffn_backward_ws_size(4, T, k, H, I, E)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty(T, H, device="cuda"), torch.empty(T, k, device="cuda")
    M.moe_expert_ffn_backward(4, layer.table, off, act, src, dst, w, x, BF16, None, dy, BF16, T, k, H, I, E,
                              layer.shared, dx, F32, dw, 0, ws, n)
    torch.cuda.synchronize()
    assert M.moe_device_error() == 0
    at = np.array([0, 1, 4095, 65536, T // 2, T - 2, T - 1])
    pick = lambda t: t[torch.from_numpy(at).cuda()].double().cpu().numpy()      # noqa: E731
    rx, rw, ex, ew = R.experts_backward(4, H, I, blobs, blobs[0], pick(ids).astype(int), pick(w), pick(x), pick(dy),
                                        R.U16)
    assert (np.abs(pick(dx) - rx) <= ex).all() and (np.abs(pick(dw) - rw) <= ew).all()


@pytest.mark.parametrize("bits", [2, 4])
@pytest.mark.parametrize("T,k,E", [(64, 10, 160), (700, 8, 40)])
def test_expert_backward_with_full_pipelines(bits, T, k, E):
    """Many long tiles a block, so that every ring of stages is in use at once:
    the two forms agree on every row, and no run differs from another."""
    H, I = 2048, 512
    c = _Case(bits, T, k, H, I, E, True, 29, sigma=0.02)
    want = c.run(M.MOE_Q8, BF16, F32, M.MOE_MODE_GEMV)
    runs = [c.run(M.MOE_Q8, BF16, F32, M.MOE_MODE_GEMM) for _ in range(6)]
    assert M.moe_device_error() == 0
    # about ten roundings of half a step along a value's path, independent of each other, as in `check`
    rms = np.sqrt(10.0) * (R.U16 + 32 * R.U32)
    for got, ref in zip(runs[0], want):
        off = torch.linalg.norm((got - ref).double(), dim=-1) / torch.linalg.norm(ref.double(), dim=-1)
        assert torch.linalg.norm((got - ref).double()) <= rms * torch.linalg.norm(ref.double())
        if got is runs[0][0]:
            assert (off <= 2 * rms).all(), off.max()               # a row's 2048 values: within a factor of the whole's
    for dx, dw in runs[1:]:
        assert torch.equal(dx, runs[0][0]) and torch.equal(dw, runs[0][1])


def test_expert_backward_wait_timeout_recovers():
    """A pipeline wait that runs out sets the error word and leaves the next call exact."""
    c = _Case(4, 200, 2, 512, 256, 8, True, 28)
    want = c.run(F32, F32, F32, M.MOE_MODE_GEMM)
    M.moe_test_hook(M.MOE_HOOK_WAIT_LIMIT_NS, 1)
    try:
        c.run(F32, F32, F32, M.MOE_MODE_GEMM)
        assert M.moe_device_error() & M.MOE_DEVERR_TIMEOUT
    finally:
        M.moe_test_hook(M.MOE_HOOK_WAIT_LIMIT_NS, 0)
    got = c.run(F32, F32, F32, M.MOE_MODE_GEMM)
    assert M.moe_device_error() == 0
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


# ----------------------------------------------------------------- router
def _router_case(T, H, E, dld, xd, wd, seed):
    rng = np.random.default_rng(seed)
    dl = _dev((rng.standard_normal((T, E)) / 16).astype(np.float32)).to(_tt(dld))
    x = _dev(rng.standard_normal((T, H)).astype(np.float32)).to(_tt(xd))
    w = _dev((0.1 * rng.standard_normal((E, H))).astype(np.float32)).to(_tt(wd))
    return dl, x, w, _dev((0.1 * rng.standard_normal((T, H))).astype(np.float32))


ROUTER = [(1, 8, 1), (3, 64, 7), (64, 128, 64), (65, 136, 40), (200, 256, 16), (129, 264, 130), (77, 64, 1100),
          (1000, 128, 24), (4100, 64, 8), (300, 72, 512)]


@pytest.mark.parametrize("T,H,E", ROUTER)
@pytest.mark.parametrize("dld,xd,wd", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16)])
def test_router_backward(T, H, E, dld, xd, wd):
    dl, x, w, add = _router_case(T, H, E, dld, xd, wd, T + H + E)
    d, xv, wv, av = (t.double().cpu().numpy() for t in (dl, x, w, add))
    n = M.moe_router_backward_ws_size(T, H, E, dld, xd, wd)
    ws = torch.full((max(16, n),), 255, dtype=torch.uint8, device="cuda")
    for dxd in (F32, BF16):
        for dx_in in (None, add):
            dx, dw = _guarded(T * H, _tt(dxd), 6.0), _guarded(E * H, _tt(wd), 6.0)
            db = _guarded(E, torch.float32, 6.0)
            M.moe_router_backward(dl, dld, x, xd, w, wd, dx_in, T, H, E, dx, dxd, dw, db, ws, n)
            torch.cuda.synchronize()
            assert M.moe_device_error() == 0
            for out, cnt in ((dx, T * H), (dw, E * H), (db, E)):
                assert (out[cnt:] == 6.0).all()
            # fp32 sums of n products: at most (n + 2) steps of half a unit on the sum of magnitudes; a
            # tensor core may cut instead of round, twice that
            def close(got, want, size, terms, half):
                b = 2 * (terms + 4) * R.U32 * size
                err = np.abs(got.double().cpu().numpy() - want)
                assert (err <= b + half * (np.abs(want) + b) * 1.01 + 1e-37).all(), (err / (b + 1e-30)).max()
            base = 0 if dx_in is None else av
            close(dx[:T * H].view(T, H), d @ wv + base, np.abs(d) @ np.abs(wv) + np.abs(base), E, _half(dxd))
            close(dw[:E * H].view(E, H), d.T @ xv, np.abs(d).T @ np.abs(xv), T, _half(wd))
            close(db[:E], d.sum(0), np.abs(d).sum(0), T, R.U32)
    # one output at a time gives the same values
    dx1, dw1, db1 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    M.moe_router_backward(dl, dld, None, xd, w, wd, add, T, H, E, dx1, dxd, None, None, ws, n)
    M.moe_router_backward(dl, dld, x, xd, None, wd, None, T, H, E, None, dxd, dw1, None, ws, n)
    M.moe_router_backward(dl, dld, None, xd, None, wd, None, T, H, E, None, dxd, None, db1, ws, n)
    assert torch.equal(dx1[:T * H], dx[:T * H]) and torch.equal(dw1[:E * H], dw[:E * H]) and torch.equal(db1[:E], db[:E])


def test_router_backward_in_place_and_without_tokens():
    T, H, E = 130, 256, 64
    dl, x, w, add = _router_case(T, H, E, BF16, BF16, BF16, 5)
    n = M.moe_router_backward_ws_size(T, H, E, BF16, BF16, BF16)
    ws = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, H, device="cuda")
    M.moe_router_backward(dl, BF16, x, BF16, w, BF16, add, T, H, E, out, F32, None, None, ws, n)
    M.moe_router_backward(dl, BF16, x, BF16, w, BF16, add, T, H, E, add, F32, None, None, ws, n)
    assert torch.equal(out, add)
    dw, db = torch.ones(E, H, dtype=torch.bfloat16, device="cuda"), torch.ones(E, device="cuda")
    M.moe_router_backward(None, BF16, None, BF16, w, BF16, None, 0, H, E, None, F32, dw, db, ws, n)
    assert (dw == 0).all() and (db == 0).all()


def test_router_backward_wait_timeout_recovers():
    T, H, E = 700, 512, 128
    dl, x, w, add = _router_case(T, H, E, BF16, BF16, BF16, 6)
    n = M.moe_router_backward_ws_size(T, H, E, BF16, BF16, BF16)
    ws = torch.empty(max(16, n), dtype=torch.uint8, device="cuda")

    def run():
        dx, dw, db = torch.empty(T, H, device="cuda"), torch.empty_like(w), torch.empty(E, device="cuda")
        M.moe_router_backward(dl, BF16, x, BF16, w, BF16, add, T, H, E, dx, F32, dw, db, ws, n)
        torch.cuda.synchronize()
        return dx, dw, db
    want = run()
    M.moe_test_hook(M.MOE_HOOK_WAIT_LIMIT_NS, 1)
    try:
        run()
        assert M.moe_device_error() & M.MOE_DEVERR_TIMEOUT
    finally:
        M.moe_test_hook(M.MOE_HOOK_WAIT_LIMIT_NS, 0)
    got = run()
    assert M.moe_device_error() == 0 and all(torch.equal(a, b) for a, b in zip(want, got))


# ------------------------------------------------- the calls in one step
@pytest.mark.parametrize("wdt,T,mode", [("bf16", 5, 0), ("bf16", 150, 0), ("f32", 70, 0), ("bf16", 40, M.MOE_MODE_GEMV)])
def test_train_step(wdt, T, mode):
    """forward() and backward() of one layer: every gradient against the
    64-bit chain on the same routing and checkpoint."""
    H, I, E, k = 256, 128, 24, 3
    lay = W.make_layer(7, 4, H, I, E, k, shared=True, w_dtype=wdt)
    g = M.MoELayer(4, H, I, E, k, lay.blobs, lay.shared, lay.w_router, wdt)
    x = W.bf16_bits_to_f32(W.make_tokens(8, T, H, "bf16")).astype(np.float32)
    rng = np.random.default_rng(T)
    dy = rng.standard_normal((T, H)).astype(np.float32)
    mask = np.ones(T, np.uint8)
    mask[1::4] = 0
    dy[mask == 0] = 0
    b, z, dl = 0.5, 0.01, 2.0
    step = M.TrainStep(g, T, BF16, dy_dtype=F32, mode=mode, balance_coef=b, z_coef=z)
    with pytest.raises(RuntimeError, match="forward"):
        step.backward(_dev(dy))
    y, loss = step.forward(_dev(x).bfloat16(), token_mask=_dev(mask))
    out = step.backward(_dev(dy), d_loss=torch.tensor([dl], device="cuda"))
    torch.cuda.synchronize()
    assert M.moe_device_error() == 0
    plain = g.forward(_dev(x).bfloat16(), BF16, mode=mode)
    assert torch.equal(plain.y[:T * H].view(T, H), y)                 # the forward pass is the layer's own
    ids = step.bufs.ids[:T * k].cpu().numpy().reshape(T, k)
    w = step.bufs.w[:T * k].cpu().numpy().reshape(T, k)
    logits = step.bufs.logits[:T * E].cpu().numpy().reshape(T, E)
    counts, losses, lgrad = R.balance(logits, ids, mask, E, b, z)
    assert np.array_equal(step.counts.cpu().numpy(), counts)
    assert np.allclose(loss.cpu().numpy(), losses, rtol=1e-5)          # the call's own test has the bound
    xv = R.act8(x)[2]
    gemm = not (mode == M.MOE_MODE_GEMV or T <= 4)
    dx, dw, ex, ew = R.experts_backward(4, H, I, lay.blobs, lay.shared, ids, w, xv, dy.astype(np.float64),
                                        R.U16 if gemm else 0.0)
    want_dl = dl * lgrad + R.gates(ids, w, dw, E, mask != 0)
    wr = (W.bf16_bits_to_f32(lay.w_router) if wdt == "bf16" else lay.w_router).astype(np.float64)
    # errors of d_logits: the gates' (through dw), rounding to its type, fp32 noise of the loss term
    edw = np.zeros((T, E))
    for t in range(T):
        if mask[t]:
            np.add.at(edw[t], ids[t], w[t] * (ew[t] + (w[t] * ew[t]).sum()) + 40 * R.U32 * np.abs(w[t] * dw[t]))
    half = R.UBF if wdt == "bf16" else R.U32
    edl = edw + 1e-4 * np.abs(dl * lgrad) + half * np.abs(want_dl) * 1.01 + 1e-9
    gdl = step.d_logits.double().cpu().numpy()
    assert (np.abs(gdl - want_dl) <= edl).all()
    # the router's products from the d_logits it was given: only their own errors
    sums = 2 * (max(E, T) + 4) * R.U32
    want = gdl.T @ xv
    b1 = sums * (np.abs(gdl).T @ np.abs(xv))
    assert (np.abs(out["d_w_router"].double().cpu().numpy() - want) <= b1 + half * 1.01 * (np.abs(want) + b1) + 1e-30).all()
    assert (np.abs(out["d_bias"].double().cpu().numpy() - gdl.sum(0)) <= sums * np.abs(gdl).sum(0) + 1e-30).all()
    want = dx + gdl @ wr
    b2 = ex + sums * (np.abs(gdl) @ np.abs(wr) + np.abs(dx))
    assert (np.abs(out["dx"].double().cpu().numpy() - want) <= b2 + R.UBF * 1.01 * (np.abs(want) + b2)).all()


@pytest.mark.parametrize("T", [2, 48])
def test_train_step_in_a_graph_and_two_in_flight(T):
    """Two steps (two layers of a model) captured together and replayed on new
    inputs give what eager calls give; each owns its buffers."""
    H, I, E, k = 256, 128, 16, 2
    layers = []
    for s in (1, 2):
        lay = W.make_layer(s, 4, H, I, E, k, shared=True, w_dtype="bf16")
        layers.append(M.MoELayer(4, H, I, E, k, lay.blobs, lay.shared, lay.w_router, "bf16"))
    x = torch.randn(T, H, device="cuda").bfloat16()
    dy = torch.randn(T, H, device="cuda")

    def steps():
        return [M.TrainStep(g, T, BF16, balance_coef=0.1, z_coef=0.01) for g in layers]

    def run(ss):
        y0, _ = ss[0].forward(x)
        ss[1].forward(y0.bfloat16())
        o1 = ss[1].backward(dy)
        o0 = ss[0].backward(o1["dx"].float())
        return [o0["dx"], o0["d_w_router"], o0["d_bias"], o1["dx"], o1["d_w_router"], o1["d_bias"]]
    captured = steps()
    run(captured)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs = run(captured)
    for seed in (3, 4):
        torch.manual_seed(seed)
        x.copy_(torch.randn(T, H, device="cuda"))
        dy.copy_(torch.randn(T, H, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, run(steps())):
            assert torch.equal(a, b) and torch.isfinite(a.float()).all()
    assert M.moe_device_error() == 0


def test_steps_on_two_streams_at_once():
    """Two steps with their own buffers, enqueued on two streams without a wait between them."""
    H, I, E, k, T = 256, 128, 16, 2, 300
    lay = W.make_layer(5, 4, H, I, E, k, shared=True, w_dtype="bf16")
    g = M.MoELayer(4, H, I, E, k, lay.blobs, lay.shared, lay.w_router, "bf16")
    steps = [M.TrainStep(g, T, BF16, balance_coef=0.1) for _ in range(2)]
    xs = [torch.randn(T, H, device="cuda").bfloat16() for _ in range(2)]
    dys = [torch.randn(T, H, device="cuda") for _ in range(2)]
    want = []
    for st, x, dy in zip(steps, xs, dys):
        st.forward(x)
        want.append([v.clone() for v in st.backward(dy).values()])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for st, x, dy, s in zip(steps, xs, dys, streams):
            st.forward(x, stream=s)
            st.backward(dy, stream=s)
    torch.cuda.synchronize()
    assert M.moe_device_error() == 0
    for st, w in zip(steps, want):
        got = [st.dx, st.d_w_router, st.d_bias]
        assert all(torch.equal(a, b) for a, b in zip(got, w))


def test_wrappers_refuse_wrong_tensors():
    x = torch.zeros(4, 64, device="cuda")
    q, s = torch.zeros(4, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, 2, dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        M.moe_act_pack8(torch.zeros(64, 4, device="cuda").t(), F32, 4, 64, q, s)
    with pytest.raises(ValueError, match="type"):
        M.moe_act_pack8(x, BF16, 4, 64, q, s)
    with pytest.raises(ValueError, match="holds"):
        M.moe_act_pack8(x, F32, 5, 64, q, s)
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.moe_act_pack8(x.cpu(), F32, 4, 64, q, s)
    with pytest.raises(M.MoEError, match="aligned"):
        M.moe_act_pack8(torch.zeros(4 * 64 + 1, device="cuda")[1:], F32, 4, 64, q, s)
