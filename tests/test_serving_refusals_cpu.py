"""Further refusals of the serving building blocks, and host-side rules of theirs (no GPU)."""
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
