"""armt_block_sync_status: one error word for all building blocks, read without touching anything else."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from recurrent_memory_transformer_gb300 import armt as B  # noqa: E402
from recurrent_memory_transformer_gb300 import build as build_mod  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FRESH = r"""
import sys
sys.path.insert(0, sys.argv[1])
import torch
from recurrent_memory_transformer_gb300 import armt as B
B.load_library()
a, b = torch.zeros(1, 128, 64, device="cuda").bfloat16(), torch.zeros(1, 256, 64, device="cuda").bfloat16()
c = torch.empty(1, 128, 256, device="cuda")
B.armt_grouped_gemm_bf16(a, b, c)
torch.cuda.synchronize()
before = torch.cuda.mem_get_info()[0]
B.armt_block_sync_status()
print(before - torch.cuda.mem_get_info()[0])
"""


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.load_library()


def test_the_first_status_of_a_process_allocates_nothing():
    """As its documentation says.  (That it brings in no kernels that were never called shows in its time alone: 50 us, 1.3 ms
    with an error word in the paged attention's modules.)"""
    out = subprocess.run([sys.executable, "-c", FRESH, ROOT], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert int(out.stdout.split()[-1]) == 0


def test_a_wait_that_gave_up_is_reported_once_whichever_block_it_was(monkeypatch):
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = B.KvCache.allocate(80, 16, 2, 64)
    a, b = torch.randn(1, 128, 64, device="cuda").bfloat16(), torch.randn(1, 256, 64, device="cuda").bfloat16()
    want, got = torch.empty(1, 128, 256, device="cuda"), torch.empty(1, 128, 256, device="cuda")
    B.armt_grouped_gemm_bf16(a, b, want)
    B.armt_block_sync_status()
    for new in (1, 7, 200):                                  # one call for each of the attention's kernels
        batch = B.PagedBatch(torch.tensor([0, new], **i32), torch.tensor([1200], **i32),
                             torch.arange(75, **i32).view(1, 75), new, new)
        q = torch.randn(new, 8, 64, device="cuda").bfloat16()
        out = torch.empty_like(q)
        workspace = B.paged_attention_workspace(cache, batch, 8)
        monkeypatch.setenv("ARMT_WAIT_LIMIT_MS", "30")
        monkeypatch.setenv("ARMT_TEST_STALL_AFTER", "1")
        B.armt_paged_attention_bf16(q, cache, batch, out, workspace)
        with pytest.raises(B.ArmtError) as e:
            B.armt_block_sync_status()
        assert e.value.status == 6
        monkeypatch.delenv("ARMT_WAIT_LIMIT_MS")
        monkeypatch.delenv("ARMT_TEST_STALL_AFTER")
        B.armt_block_sync_status()
        B.armt_paged_attention_bf16(q, cache, batch, out, workspace)
        B.armt_grouped_gemm_bf16(a, b, got)
        B.armt_block_sync_status()
        assert (out == 0).all() and torch.equal(got, want)   # (values of a fresh cache: zeros)
