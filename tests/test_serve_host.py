"""Host side of the calls around the recall: struct layouts against the header,
calls without a context, and the 64-bit definitions the GPU tests use."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import serve_ref as ref
from paged_kv_cache_meank_gb300 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_abi.LIB_PATH):
        from paged_kv_cache_meank_gb300 import build
        build.build()
    return _abi.load()


def test_calls_reject_null_context(lib):
    n0 = lib.kvm_launch_count()
    assert lib.kvm_qk_norm_rope(None, 1, None, None, 0, None, 0, None, None, 1e-6, None, None, None,
                                None, None) == -1
    assert lib.kvm_append_kv(None, None, None, 0, None, 0, None, 0, None, None, None) == -1
    assert lib.kvm_attend(None, None, None, 0, None, 0, 1.0, 1, None, 0, None, None) == -1
    assert lib.kvm_build_index_scaled(None, None, None, 0, 1, None, None, None) == -1
    assert lib.kvm_launch_count() == n0


def test_struct_layouts_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"kvm_cache": _abi.KvmCache, "kvm_batch": _abi.KvmBatch}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "kvm.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        lines += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run([cc, "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for cls in structs.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def test_the_definitions():
    # e4m3 rounding: torch's own, over every sign, tie and subnormal step
    x = torch.cat((torch.linspace(-448, 448, 20001), torch.linspace(-0.1, 0.1, 20001))).double()
    assert torch.equal(ref.encode(x), x.float().to(torch.float8_e4m3fn).view(torch.uint8))
    # scales: least power of two, at, just above and far from the border
    for most in (316.75, 448.0):
        for e in (-100, -20, 0, 7):
            assert ref.scale_for(most * 2.0 ** e, most) == 2.0 ** e
            assert ref.scale_for(most * 2.0 ** e * 1.0001, most) == 2.0 ** (e + 1)
    assert ref.scale_for(0.0, 448.0) == 2.0 ** -100 and ref.scale_for(1e-40, 448.0) == 2.0 ** -100
    # no rotation of an entry within 316.75 leaves e4m3's range
    assert 316.75 * 2 ** 0.5 < 448
    # attention: two keys by hand, an empty row
    q = torch.tensor([[1.0, 0.0], [0.0, 2.0]]).double()
    k, v = torch.tensor([[1.0, 0.0], [0.0, 1.0]]).double(), torch.tensor([[1.0, 2.0], [3.0, 4.0]]).double()
    o, lse, _ = ref.attention(q, k, v, 1.0, 0, True)
    assert torch.allclose(o[0], v[0]) and abs(float(lse[0]) - 1.0) < 1e-12
    w = torch.softmax(torch.tensor([0.0, 2.0]).double(), 0)
    assert torch.allclose(o[1], w @ v)
    o, lse, _ = ref.attention(q, k, v, 1.0, -1, True)
    assert not o[0].any() and lse[0] == -float("inf") and torch.allclose(o[1], v[0])
    # rotation at 0 is nothing, at p then -p too
    x = torch.randn(5, 8).double()
    pos = torch.arange(5)
    assert torch.allclose(ref.rotate(ref.rotate(x, pos, 1e4), pos, 1e4, -1.0), x)
