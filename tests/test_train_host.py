"""CPU checks of the training side's host code: where a workspace's parts lie,
and what TrainStep does before it launches anything."""
import ctypes as C
import subprocess

import numpy as np

import quantized_expert_ffn_route_b200 as M

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
