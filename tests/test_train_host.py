"""CPU checks of the training side's host code: where a workspace's parts lie,
and what TrainStep does before it launches anything."""
import contextlib
import ctypes as C
import subprocess

import pytest
import torch

import quantized_expert_ffn_route_b200 as M
from quantized_expert_ffn_route_b200 import train

CSRC = M.LIB_PATH.parent.parent / "csrc"


def _host_lib(tmp_path, name, body):
    """A host library of a few lines that include the library's own headers."""
    src, so = tmp_path / f"{name}.cpp", tmp_path / f"{name}.so"
    src.write_text(body)
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o", str(so)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return C.CDLL(str(so))


# ------------------------------------------------------------- workspaces
def test_workspace_parts_are_aligned_wherever_it_starts(tmp_path):
    """Any 16-byte aligned workspace: its parts start at a multiple of 256 (a
    tensor map in global memory needs 128) and end within the size that the
    call asks for."""
    lib = _host_lib(tmp_path, "ws", '#include "train/ws.h"\n'
                    'extern "C" size_t start(size_t p) { return (size_t)moe::ws_start((void *)p); }\n'
                    'extern "C" size_t align() { return moe::kWsAlign; }\n'
                    'extern "C" size_t slack() { return moe::kWsSlack; }\n')
    for f in (lib.start, lib.align, lib.slack):
        f.restype = C.c_size_t
    lib.start.argtypes = [C.c_size_t]
    align, slack = lib.align(), lib.slack()
    assert align % 128 == 0
    for base in (1 << 12, (1 << 40) + 512, (1 << 47) - 4096):
        for p in range(base, base + 2 * align, 16):
            at = lib.start(p)
            assert at % align == 0 and p <= at <= p + slack
    # the parts are whole multiples of the alignment; what the start may take comes on top
    for bits, T, k, H, I, E in ((4, 1, 1, 128, 128, 1), (2, 7, 3, 384, 128, 5), (4, 777, 3, 1152, 384, 40)):
        assert M.moe_expert_ffn_backward_ws_size(bits, T, k, H, I, E, M.MOE_MODE_GEMM) % align == slack % align


# -------------------------------------------------------------- TrainStep
class _Reached(Exception):
    """The layer's forward pass, which launches kernels, was called."""


class _StandIn:
    """A layer without memory: what TrainStep reads of one."""

    def __init__(self, device="meta"):
        self.bits, self.H, self.I, self.E, self.k = 4, 256, 128, 16, 2
        self.device = torch.device(device)
        self.arena = torch.empty(16, dtype=torch.uint8, device="meta")
        self.table = torch.empty(self.E, dtype=torch.int64, device="meta")
        self.shared = None
        self.w_dtype = M.MOE_BF16
        self.w_router = torch.empty(self.E, self.H, dtype=torch.bfloat16, device="meta")
        self.bias = None

    def forward(self, *args, **kw):
        raise _Reached


class _FakeCuda(torch.Tensor):
    """A host tensor that says it lies on a CUDA device (nothing may read it)."""

    @staticmethod
    def __new__(cls, t, index=0):
        r = torch.Tensor._make_subclass(cls, t)
        r.index_ = index
        return r

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index_))

    def get_device(self):
        return self.index_


@pytest.fixture
def no_device_switch(monkeypatch):
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())


T = 6


def _step(**kw):
    s = M.TrainStep(_StandIn(), T, M.MOE_BF16, **kw)
    s._ran = True                                          # a good forward() went before
    return s


BAD_X = {
    "short": lambda: _FakeCuda(torch.zeros(T - 1, 256, dtype=torch.bfloat16)),
    "type": lambda: _FakeCuda(torch.zeros(T, 256)),
    "host": lambda: torch.zeros(T, 256, dtype=torch.bfloat16),
    "strided": lambda: _FakeCuda(torch.zeros(256, T, dtype=torch.bfloat16).t()),
    "no tensor": lambda: [0.0] * (256 * T),
}


@pytest.mark.parametrize("coef", [0.0, 0.5])
@pytest.mark.parametrize("bad", BAD_X)
def test_train_step_refuses_x_before_it_launches(bad, coef, no_device_switch):
    step = _step(balance_coef=coef)
    with pytest.raises((ValueError, TypeError), match="TrainStep.forward: x"):
        step.forward(BAD_X[bad]())
    with pytest.raises(RuntimeError, match="forward"):     # the last step's state is no longer whole
        step.backward(_FakeCuda(torch.zeros(T, 256)))


@pytest.mark.parametrize("coef", [0.0, 0.5])
@pytest.mark.parametrize("mask", [lambda: _FakeCuda(torch.ones(T - 1, dtype=torch.uint8)),
                                  lambda: _FakeCuda(torch.ones(T)), lambda: torch.ones(T, dtype=torch.bool)])
def test_train_step_refuses_a_mask_before_it_launches(mask, coef, no_device_switch):
    step = _step(balance_coef=coef)
    with pytest.raises(ValueError, match="TrainStep.forward: token_mask"):
        step.forward(_FakeCuda(torch.zeros(T, 256, dtype=torch.bfloat16)), token_mask=mask())
    with pytest.raises(RuntimeError, match="forward"):
        step.backward(_FakeCuda(torch.zeros(T, 256)))


def test_train_step_without_a_whole_forward_has_no_backward(no_device_switch):
    """A forward pass that fails on its way leaves nothing to go back from."""
    step = _step()
    with pytest.raises(_Reached):                          # good arguments reach the layer
        step.forward(_FakeCuda(torch.zeros(T + 1, 256, dtype=torch.bfloat16)),
                     token_mask=_FakeCuda(torch.ones(T, dtype=torch.bool)))
    with pytest.raises(RuntimeError, match="forward"):
        step.backward(_FakeCuda(torch.zeros(T, 256)))


def test_train_step_lies_on_its_layers_device(monkeypatch):
    """A layer on "cuda" (no index) lies where its arena does, whichever device
    is current when the step is made: every buffer goes there, and sizes, which
    follow the device, are asked for there."""
    inside = []

    @contextlib.contextmanager
    def device(d):
        inside.append(torch.device(d))
        yield
        inside.pop()
    monkeypatch.setattr(torch.cuda, "device", device)
    asked = []
    for mod, name in [(train, n) for n in train.SIGNATURES if n.endswith("_ws_size")] + [
            (M, n) for n in ("moe_route_ws_size", "moe_permute_ws_size", "moe_expert_ffn_ws_size")]:
        def ask(*a, real=getattr(mod, name), name=name):
            asked.append(name)
            assert inside == [torch.device("meta")], name
            return real(*a)
        monkeypatch.setattr(mod, name, ask)
    step = M.TrainStep(_StandIn("cuda"), T, M.MOE_BF16, balance_coef=0.5)
    assert len(set(asked)) == 6 and not inside
    found = [v for o in (step, step.bufs) for v in vars(o).values() if isinstance(v, torch.Tensor)]
    assert len(found) > 20 and all(v.device.type == "meta" for v in found)
