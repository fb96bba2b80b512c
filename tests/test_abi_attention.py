"""The C ABI of the attention operators, checked on the CPU: struct layouts,
host-only size helpers and NULL handles."""
import ctypes
import os
import subprocess

import pytest

from tile_centric_comm_gb300 import build as tdg_build
from tile_centric_comm_gb300 import tdg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STRUCTS = {"tdg_paged_cache": tdg.PagedCacheDesc, "tdg_rope_append_args": tdg.RopeAppendArgs,
           "tdg_prompt_attention_args": tdg.PromptAttentionArgs, "tdg_paged_decode_args": tdg.PagedDecodeArgs}


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


def test_sizes(L):
    assert tdg.paged_pool_bytes(10, 64, 8, 128) == 10 * 64 * 8 * 128 * 2
    assert tdg.paged_pool_bytes(10, 16, 3, 64, e4m3=True) == 10 * 16 * 3 * 64
    for bad in ((0, 64, 8, 128), (-1, 64, 8, 128), (10, 48, 8, 128), (10, 512, 8, 128), (10, 64, 0, 128), (10, 64, 8, 96)):
        assert tdg.paged_pool_bytes(*bad) == 0
    assert L.tdg_paged_pool_bytes(10, 64, 8, 128, 2) == 0
    assert tdg.paged_decode_part_bytes(64, 8, 128) >= 2 * 152 * 16 * 130 * 4
    assert tdg.paged_decode_part_bytes(64, 8, 64) < tdg.paged_decode_part_bytes(64, 8, 128) < 32 << 20
    for bad in ((0, 8, 128), (9, 8, 128), (129, 1, 128), (64, 8, 96)):
        assert tdg.paged_decode_part_bytes(*bad) == 0


def test_null_handles(L):
    assert L.tdg_rope_append(None, None, None) == tdg.TDG_ERR_INVALID
    assert L.tdg_prompt_attention(None, None, None) == tdg.TDG_ERR_INVALID
    assert L.tdg_paged_decode(None, None, None) == tdg.TDG_ERR_INVALID


def test_packed_arguments_match_the_structures():
    """The binding packs arguments with one struct call: same layout as the structures."""
    import random

    def values(cls):
        for name, kind in cls._fields_:
            if isinstance(kind, type) and issubclass(kind, ctypes.Structure):
                yield from values(kind)
            elif hasattr(kind, "_length_"):
                yield from (random.randrange(1, 1 << 20) for _ in range(kind._length_))
            elif kind is ctypes.c_float:
                yield 0.25
            else:
                yield random.randrange(1, 1 << 20)

    def fill(obj, it):
        for name, kind in obj._fields_:
            if isinstance(kind, type) and issubclass(kind, ctypes.Structure):
                fill(getattr(obj, name), it)
            elif hasattr(kind, "_length_"):
                for i in range(kind._length_):
                    getattr(obj, name)[i] = next(it)
            else:
                setattr(obj, name, next(it))

    for cls, pack in ((tdg.RopeAppendArgs, tdg._pack_rope), (tdg.PromptAttentionArgs, tdg._pack_prompt),
                      (tdg.PagedDecodeArgs, tdg._pack_decode)):
        v = list(values(cls))
        obj = cls()
        fill(obj, iter(v))
        assert pack(*v) == bytes(obj), cls.__name__
