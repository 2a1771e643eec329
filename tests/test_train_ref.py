"""CPU checks of the training side: the plain definitions' gradients against
differences, the 8-bit format's properties, and every refusal of the calls."""
import ctypes as C
import re
import subprocess

import numpy as np
import pytest

import quantized_expert_ffn_route_b200 as M
import workloads as W
from tests import train_ref as R


# ------------------------------------------------------------ definitions
def _difference(f, x, h):
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


@pytest.mark.parametrize("masked", [False, True])
def test_balance_gradient_matches_differences(masked):
    rng = np.random.default_rng(1)
    T, E, k = 5, 7, 2
    l = rng.standard_normal((T, E))
    ids = np.argsort(-l, 1, kind="stable")[:, :k]
    mask = np.array([1, 0, 1, 1, 0]) if masked else None
    got = R.balance(l, ids, mask, E, 0.7, 0.3)[2]
    # central differences of step h: error about h^2 (third derivative, O(1)) + 1e-16 / h
    want = _difference(lambda v: R.balance(v, ids, mask, E, 0.7, 0.3)[1][0], l, 1e-5)
    assert np.abs(got - want).max() <= 1e-9


def test_gate_gradient_matches_differences():
    rng = np.random.default_rng(2)
    T, E, k = 3, 6, 3
    l, dw = rng.standard_normal((T, E)), rng.standard_normal((T, k))
    ids = np.argsort(-l, 1, kind="stable")[:, :k]

    def soft(v):
        s = np.exp(np.take_along_axis(v, ids, 1))
        return s / s.sum(1, keepdims=True)
    want = _difference(lambda v: (soft(v) * dw).sum(), l, 1e-5)
    assert np.abs(R.gates(ids, soft(l), dw, E) - want).max() <= 1e-9


@pytest.mark.parametrize("bits", [2, 4])
def test_expert_gradient_matches_differences(bits):
    H, I, n = 128, 128, 2
    rng = np.random.default_rng(3)
    Wt = R.matrices(bits, H, I, W.random_expert_blob(np.random.Generator(np.random.PCG64(4)), bits, H, I, 0.1))
    x, dy = rng.standard_normal((n, H)), rng.standard_normal((n, H))
    dxp, dw, _, _ = R.ffn_backward(Wt, x, dy, 0, 0)
    want = _difference(lambda v: (R.ffn_forward(Wt, v) * dy).sum(), x, 1e-5)
    assert np.abs(dxp - want).max() <= 1e-7 * max(1, np.abs(want).max())
    assert np.allclose(dw, (R.ffn_forward(Wt, x) * dy).sum(1), rtol=1e-12)


def test_act8_format():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((64, 256)) * np.exp(3 * rng.standard_normal((64, 1)))
    q, s, v = R.act8(x)
    step = np.repeat(2.0 ** (s.astype(float) - 127), 32, 1)
    amax = np.repeat(np.abs(x.reshape(64, -1, 32)).max(-1), 32, 1)
    assert np.abs(v - x).max() > 0 and (np.abs(v - x) <= step / 2).all() and (step / 2 <= amax / 127).all()
    assert (np.abs(q.reshape(64, -1, 32)).max(-1) >= 64).all()        # no smaller step would do
    assert np.array_equal(R.act8(v)[2], v)                            # values are kept exactly
    assert np.array_equal(W.bf16_bits_to_f32(W.f32_to_bf16_bits(v.astype(np.float32))), v.astype(np.float32))


# ---------------------------------------------------------------- the ABI
def _declared():
    src = re.sub(r"/\*.*?\*/", "", M.TRAIN_HEADER.read_text(), flags=re.S)
    return sorted(set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", src)))


def test_library_exports_the_training_calls():
    names = _declared()
    assert len(names) == 9
    out = subprocess.run(["nm", "-D", "--defined-only", str(M.LIB_PATH)], capture_output=True, text=True).stdout
    assert set(names) <= set(re.findall(r" T (moe_\w+)$", out, flags=re.M))
    from quantized_expert_ffn_route_b200.train import SIGNATURES
    assert set(SIGNATURES) == set(names)


@pytest.mark.parametrize("lang", ["c", "c++"])
def test_training_header_compiles_as_c_and_cpp(lang):
    r = subprocess.run(["gcc" if lang == "c" else "g++", "-fsyntax-only", "-Wall", "-Werror", "-x", lang,
                        str(M.TRAIN_HEADER)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def _buf():
    b = np.zeros(1 << 16, np.float32)
    p = (b.ctypes.data + 255) // 256 * 256
    return b, p


def _refused(name, args, changes):
    """Each change (position -> value) of a good argument list is refused."""
    f = getattr(M.lib(), name)
    for change in changes:
        a = list(args)
        for i, v in change.items():
            a[i] = v
        assert f(*a) == M.MOE_EINVAL, (name, change)
        assert M.moe_last_error() != ""


def test_act8_refusals():
    _, p = _buf()
    bad = [{1: 7}, {1: M.MOE_Q8}, {2: -1}, {3: 0}, {3: 48}, {0: None}, {4: None}, {5: None}, {0: p + 8}, {4: p + 4},
           {5: p + 1}, {4: p}]
    q = p + 4096
    _refused("moe_act_pack8", [p, 0, 4, 64, q, q, None], bad)
    _refused("moe_act_unpack8", [q, q, 4, 64, p, 0, None],
             [{5: 7}, {5: 2}, {2: -1}, {3: 16}, {0: None}, {1: None}, {4: None}, {0: p + 8}, {1: p + 8}, {4: p + 8},
              {0: p}])
    assert M.lib().moe_act_pack8(None, 0, 0, 64, None, None, None) == M.MOE_OK
    assert M.lib().moe_act_unpack8(None, None, 0, 64, None, 1, None) == M.MOE_OK


def test_balance_refusals():
    _, p = _buf()
    n = M.moe_balance_ws_size(4, 16)
    assert n > 0 and M.moe_balance_ws_size(0, 16) == 0 and M.moe_balance_ws_size(4, 0) == 0
    good = [p, p, None, 4, 16, 2, 1.0, 0.0, p, p, p, n, None]
    _refused("moe_balance_loss", good,
             [{3: -1}, {4: 0}, {4: 32769}, {5: 0}, {5: 17}, {5: 33, 4: 64}, {3: 1 << 30, 5: 2}, {0: None}, {1: None},
              {8: None}, {9: None}, {10: None}, {11: n - 1}, {0: p + 4}, {1: p + 4}, {8: p + 4}, {9: p + 4}, {10: p + 8}])
    good = [p, p, p, p, None, p, None, 4, 16, 2, 1.0, 0.0, p + 4096, 0, None]
    _refused("moe_route_backward", good,
             [{7: -1}, {8: 0}, {9: 0}, {9: 17}, {13: 2}, {13: -1}, {12: None}, {12: p + 4}, {2: None}, {3: None},
              {0: None}, {1: None}, {0: p + 4}, {2: p + 4}, {3: p + 8}, {5: p + 4}, {6: p + 2}, {12: p}])
    assert M.lib().moe_route_backward(*([None] * 7), 0, 16, 2, 1.0, 0.0, None, 0, None) == M.MOE_OK


def test_expert_backward_refusals():
    _, p = _buf()
    T, k, H, I, E = 4, 2, 256, 128, 16
    n = M.moe_expert_ffn_backward_ws_size(4, T, k, H, I, E, M.MOE_MODE_GEMV)
    assert n > 0 and M.moe_expert_ffn_backward_ws_size(3, T, k, H, I, E) == 0
    assert M.moe_expert_ffn_backward_ws_size(4, 0, k, H, I, E) == 0
    q = p + 4096
    #       bits blobs offs act src dst w  x  xd xs    dy dyd T  k  H  I  E  shared dx dxd dw mode ws n
    good = [4, p, p, p, p, p, p, p, 0, None, p, 0, T, k, H, I, E, None, q, 0, p, 1, p, n, None]
    _refused("moe_expert_ffn_backward", good,
             [{0: 3}, {12: -1}, {13: 0}, {13: 17}, {13: 33, 16: 64}, {14: 200}, {14: 8320}, {15: 64}, {15: 4224}, {16: 0},
              {21: 3}, {21: -1}, {8: 3}, {8: 2}, {9: p}, {11: 2}, {19: 2}, {22: None}, {23: n - 1}, {18: p},
              {12: 1 << 30}] +
             [{i: None} for i in (1, 2, 3, 4, 5, 6, 7, 10, 18, 20)] +
             [{i: p + 8} for i in (1, 2, 3, 4, 5, 6, 7, 10, 17, 18, 20, 22)] + [{8: 2, 9: p + 8}])
    assert M.lib().moe_expert_ffn_backward(4, *([None] * 7), 0, None, None, 0, 0, k, H, I, E, None, None, 0, None, 0,
                                           None, 0, None) == M.MOE_OK


def test_router_backward_refusals():
    _, p = _buf()
    T, H, E = 4, 64, 16
    q, r = p + 4096, p + 8192
    #       dl dld x xd w wd dx_in T H E dx dxd dw db ws n
    good = [p, 0, p, 0, p, 0, None, T, H, E, q, 0, r, r, None, 0, None]
    _refused("moe_router_backward", good,
             [{1: 2}, {3: 2}, {5: 7}, {11: 2}, {7: -1}, {8: 0}, {8: 12}, {9: 0}, {9: 32769}, {0: None}, {2: None},
              {4: None}, {10: None, 12: None, 13: None}, {10: p}, {6: q, 11: 1}, {12: p},
              {12: q}, {6: r}, {7: (1 << 30) + 1}] +
             [{i: p + 8} for i in (0, 2, 4, 6, 10, 12, 13)])
    # large bf16 products need the workspace that the size call asks for
    n = M.moe_router_backward_ws_size(8192, 2048, 512, 1, 1, 1)
    if n:
        _refused("moe_router_backward", [p, 1, p, 1, p, 1, None, 8192, 2048, 512, q, 1, r, None, p, n, None],
                 [{14: None}, {15: n - 1}, {14: p + 8}])


def test_wrappers_check_their_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        M.moe_act_pack8(x, M.MOE_F32, 4, 64, x, x)
    with pytest.raises(TypeError, match="CUDA tensor"):
        M.moe_act_pack8([0.0], M.MOE_F32, 4, 64, None, None)
    assert C.sizeof(C.c_void_p) == 8


def test_no_overlap_between_workspace_parts():
    """The workspace grows with every argument that adds rows or columns."""
    size = M.moe_expert_ffn_backward_ws_size
    base = size(4, 64, 2, 256, 128, 16, 0)
    assert size(4, 65, 2, 256, 128, 16, 0) > base and size(4, 64, 3, 256, 128, 16, 0) > base
    assert size(4, 64, 2, 384, 128, 16, 0) > base and size(4, 64, 2, 256, 256, 16, 0) > base
