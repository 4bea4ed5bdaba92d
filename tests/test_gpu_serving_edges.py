"""The serving building blocks at the ends of what their documentation allows.

Tolerances are those of test_gpu_serving.py (`Setup.check`), which hold for
any scale bytes: a weight's error there is relative to the largest weight times
value scale, and the sum of weights is exact to fp32 whatever the scales are.
One term more where weights are taken apart from the values' scales (bf16
caches, and the many-row kernel over either type), `flush`: the exponential
instruction gives 0 for results under 2^-126, and its reference is at most the
row's largest score, so a weight of w_j < 2^-126 of the largest may be lost
whole, and the output is off by at most 2^-126 sum |v_j| over such keys (the sum
of weights, at least 1 in the same unit, by n 2^-126 of itself: nothing).
Beside values of 2^100 that is far above the other terms; beside ordinary ones
far below.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from recurrent_memory_transformer_gb300 import armt as B  # noqa: E402
from recurrent_memory_transformer_gb300 import build as build_mod  # noqa: E402
from tests import plain_serving as P  # noqa: E402
from tests.test_gpu_serving import Setup  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    build_mod.build()
    B.load_library()


class Wide(Setup):
    """A Setup whose check counts lost weights."""

    def check(self, q, out, scale=None):
        lost = 0.0
        if self.type == B.CACHE_BF16 or self.max_new * (q.shape[1] // self.hkv) > (32 if self.hd == 128 else 64):
            lost = 2.0 ** -126 * np.nansum(np.abs(self.v[np.isfinite(self.v)]))
        rows = self.row_start[0], self.row_start[-1]
        ref = P.attention(q.double().cpu().numpy(), self.k, self.v, self.row_start, self.kv_len, self.table,
                          self.max_new, self.hd ** -0.5 if scale is None else scale)[0]
        got = out.double().cpu().numpy()
        off = got - ref
        less = ref + np.sign(off) * np.maximum(np.abs(off) - lost, 0.0)  # what is left to the other terms
        got[rows[0]:rows[1]] = less[rows[0]:rows[1]]
        super().check(q, torch.from_numpy(got), scale)


def set_codes(s, k=None, v=None, k_scale=None, v_scale=None):
    """Replaces an e4m3 cache's contents, and the float64 view of them."""
    c = s.cache
    for pool, x in ((c.k, k), (c.v, v)):
        if x is not None:
            pool.view(torch.uint8).copy_(torch.from_numpy(x))
    for pool, x in ((c.k_scale, k_scale), (c.v_scale, v_scale)):
        if x is not None:
            pool.copy_(torch.from_numpy(x))
    s.k, s.v = (P.e4m3_decode(pool.view(torch.uint8).cpu().numpy()) *
                np.exp2(sc.cpu().numpy().astype(np.float64) - 127)[..., None]
                for pool, sc in ((c.k, c.k_scale), (c.v, c.v_scale)))


# new rows for each of the kernels over an e4m3 cache, 4 heads a kv head: 8, 16, 32 rows, 64 (head_dim 64; with 128 the
# many-row kernel), more
ROWS = [(64, 1), (128, 2), (64, 3), (128, 4), (64, 7), (128, 8), (64, 12), (128, 12), (64, 40), (128, 40)]


@pytest.mark.parametrize("kv", [150, 7000])
@pytest.mark.parametrize("low,high", [(27, 247), (240, 247), (27, 45)])
@pytest.mark.parametrize("hd,new", ROWS)
def test_value_scales_over_their_whole_range(hd, new, low, high, kv):
    """Scale bytes of the values drawn from all the library writes, from its largest and from its smallest."""
    s = Wide("e4m3", 1, hd, 32, [new], [kv], seed=new)
    rng = s.rng
    codes = rng.integers(0, 256, s.k.shape).astype(np.uint8)
    codes[(codes & 0x7F) >= 0x60] &= 0x9F                    # |code| < 32: |v| < 2^125, no bf16 infinity
    if new * 4 > (64 if hd == 64 else 32):
        high = min(high, 227)                                # the many-row kernel: sums of bf16 products (see armt.h)
        low = min(low, high)
    set_codes(s, v=codes, v_scale=rng.integers(low, high + 1, s.k.shape[:3]).astype(np.uint8))
    q = s.queries(4)
    s.check(q, s.attend(q))
    q.mul_(8.0)
    s.check(q, s.attend(q))


@pytest.mark.parametrize("exponent", [120, 112, 60, -85, -100])
@pytest.mark.parametrize("hd,new", ROWS)
def test_many_small_weights_beside_a_large_one(hd, new, exponent):
    """One key with v = 2^e, the others 14 octaves below it in score with v = -2^(e - 2): 0.375 * 2^e when there are
    16,384 of them.  Where one reference served both sums and e was 120, they dropped out and 2^e came back."""
    n = 16384 + new
    if new * 4 > (64 if hd == 64 else 32):
        exponent = min(exponent, 100)
    s = Setup("e4m3", 1, hd, 64, [new], [n], seed=1, spare=0)
    k = np.zeros(s.k.shape, np.uint8)
    v = np.zeros(s.k.shape, np.uint8)
    v[..., ::2] = 0xA8                                       # -0.25
    v[..., 1::2] = 0x28
    page = int(s.table[0, 3])
    k[page, 0, 5, 0] = 0x50                                  # 8 in a column where the queries have 1
    v[page, 0, 5] = 0x38                                     # 1
    byte = np.full(s.k.shape[:3], 127, np.uint8)
    set_codes(s, k=k, v=v, k_scale=byte, v_scale=byte + np.uint8(exponent % 256))
    q = torch.zeros(new, 4, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = 14 * math.log(2) / 8
    out = s.attend(q, scale=scale)
    s.check(q, out, scale=scale)
    assert ((out.double() * 2.0 ** -exponent)[..., 0] - 0.375).abs().max().item() < 2.0 ** -8
