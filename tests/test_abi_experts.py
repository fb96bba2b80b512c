"""The C ABI of the 8-bit operators and the MoE gradients, checked on the CPU:
struct layouts, packed arguments, NULL handles, and the binding's checks."""
import ctypes
import os
import random
import subprocess

import pytest
import torch

from tile_centric_comm_gb300 import build as tdg_build
from tile_centric_comm_gb300 import tdg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"tdg_quantise_args": tdg.QuantiseArgs, "tdg_scaled_gemm_args": tdg.ScaledGemmArgs,
           "tdg_moe_dispatch_e4m3_args": tdg.MoeDispatchE4m3Args, "tdg_moe_combine_grad_args": tdg.MoeCombineGradArgs,
           "tdg_moe_dispatch_grad_args": tdg.MoeDispatchGradArgs}


@pytest.fixture(scope="module")
def L():
    tdg_build.build()
    return tdg.lib()


def test_struct_layouts_match_c(tmp_path):
    lines = []
    for name, cls in STRUCTS.items():
        lines.append(f'printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'printf("{name}.{f[0]} %zu\\n", offsetof({name}, {f[0]}));' for f in cls._fields_]
    prog = tmp_path / "layout.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "tdg.h"\nint main(void) {\n' + "\n".join(lines) + "\nreturn 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    got = dict(line.split() for line in out.splitlines())
    for name, cls in STRUCTS.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert int(got[f"{name}.{f[0]}"]) == getattr(cls, f[0]).offset, f"{name}.{f[0]}"


@pytest.mark.parametrize("cls,pack", [(tdg.QuantiseArgs, tdg._pack_quantise), (tdg.ScaledGemmArgs, tdg._pack_scaled),
                                      (tdg.MoeDispatchE4m3Args, tdg._pack_dispatch_e4m3), (tdg.MoeCombineGradArgs, tdg._pack_combine_grad),
                                      (tdg.MoeDispatchGradArgs, tdg._pack_dispatch_grad)])
def test_packed_arguments_match_the_structures(cls, pack):
    v = [random.randrange(1, 1 << 20) for _ in cls._fields_]
    obj = cls(**{f[0]: x for f, x in zip(cls._fields_, v)})
    assert pack(*v) == bytes(obj)


def test_null_handles(L):
    for name in ("tdg_quantise", "tdg_scaled_gemm", "tdg_moe_dispatch_e4m3", "tdg_moe_combine_grad", "tdg_moe_dispatch_grad"):
        assert getattr(L, name)(None, None, None) == tdg.TDG_ERR_INVALID


def test_matrix_checks(L):
    """What is refused before the device is looked at, native and in Python alike."""
    tdg._attn()
    cpu = torch.device("cpu")
    x = torch.zeros(4, 32, dtype=torch.float32)
    for check in (tdg._matrix, tdg._checked_matrix):
        for bad, dtype, match in (([0.0], torch.float32, "torch.Tensor"), (x, torch.bfloat16, "bfloat16"), (x[0], torch.float32, "rows, columns"),
                                  (x.t(), torch.float32, "contiguous"), (x[:, ::2], torch.float32, "contiguous")):
            with pytest.raises((TypeError, ValueError), match=match):
                check(bad, "x", dtype, cpu)
        with pytest.raises(ValueError, match="the heap is on cuda:1"):
            check(x, "x", torch.float32, torch.device("cuda", 1))


def test_matrix_checks_agree_on_what_passes(L):
    tdg._attn()
    dev = torch.device("cpu")
    # a CPU tensor's index is -1 for both; the native check compares whole devices
    x = torch.zeros(4, 32)
    for t in (x, x[:, :8], x[:1], x[1:], x[::2], x[:, :1], x[:0], x[:, :0], x[:1, 4:8], x.expand(4, 32)):
        want = (t.data_ptr(), t.shape[1] if t.shape[0] <= 1 else t.stride(0), *t.shape)
        assert tdg._matrix(t, "x", torch.float32, dev) == want
