"""GPU checks of the training calls at the edges of what their header allows:
where buffers start, the range of the weights, rows that nobody computes."""
import numpy as np
import pytest

from tests import train_ref as R

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import quantized_expert_ffn_route_b200 as M  # noqa: E402
from tests.test_gpu_train import BF16, F32, MODES, _Case, _dev, _guarded, _router_case  # noqa: E402


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
