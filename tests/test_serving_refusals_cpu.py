"""Further refusals of the serving building blocks, and host-side rules of theirs (no GPU)."""
import os
import shutil
import subprocess

import pytest

from recurrent_memory_transformer_gb300 import armt as B
from recurrent_memory_transformer_gb300 import build as build_mod
from tests.test_serving_cpu import ARG, NO_DEVICE, Call


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


@pytest.fixture(autouse=True)
def _no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("these calls carry host pointers")


@pytest.mark.parametrize("field", ["row_start", "kv_len", "page_table"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_misaligned_arrays_of_a_batch_are_refused(lib, field, off):
    c = Call()
    setattr(c.batch, field, c.p + off)
    for st in (c.write(lib), c.read(lib), c.attend(lib), c.workspace(lib)):
        assert st == ARG
    setattr(c.batch, field, c.p + 4)
    for st in (c.write(lib), c.read(lib), c.attend(lib), c.workspace(lib)):
        assert st == NO_DEVICE


def test_a_register_split_goes_by_what_the_block_is_launched_with(tmp_path):
    """Registers come in eights, so 121 to 128 of them are one launch; fewer are refused.  (256 threads at 168 and 256 at 88,
    as in the many-row kernel over e4m3 caches, use all of 512 x 128.)"""
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src = tmp_path / "a.cpp"
    src.write_text("""
#include <cstdio>
#include "register_split.h"
int main() { for (int n = 0; n <= 255; ++n) std::printf("%d", (int)armt::split_fits(n, 512, 256, 168, 88)); }
""")
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "recurrent_memory_transformer_gb300", "csrc")
    subprocess.run([cxx, "-std=c++17", "-I", csrc, str(src), "-o", str(tmp_path / "a")], check=True)
    fits = subprocess.run([str(tmp_path / "a")], check=True, capture_output=True, text=True).stdout
    assert fits == "0" * 121 + "1" * 135
