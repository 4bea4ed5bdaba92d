"""The full-attention baseline on sequences of changing length, one model after another call's workspace."""
import dataclasses

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from oracle import armt_oracle as O  # noqa: E402
from recurrent_memory_transformer_gb300 import armt as B  # noqa: E402
from recurrent_memory_transformer_gb300 import build as build_mod  # noqa: E402
from recurrent_memory_transformer_gb300 import inputs as I  # noqa: E402


def test_shorter_sequences_after_longer_ones():
    """Causal rows depend on the tokens before them alone, so every prefix gives the long call's first rows (to the same
    bound against 64 bits: other tiles, other roundings), and a length's second call equals its first bit for bit."""
    build_mod.build()
    B.load_library()
    cfg = dataclasses.replace(I.ARMT_1B, n_layers=2, vocab=4096)
    W = I.make_weights(cfg, seed=62, norm_jitter=0.1)
    m = B.Model(cfg, B.device_weight_tensors(cfg, W))
    tok = np.random.default_rng(62).integers(0, cfg.vocab, size=300).astype(np.int32)
    W64 = O.widen_weights(W)

    def plain(rounding):
        x = W64["embed"][tok]
        for l in range(cfg.n_layers):
            x = O.llama_block(x, cfg, W64, l, rounding)
        return O.rmsnorm(x, W64["norm_f"], cfg.norm_eps)
    exact = plain(O.EXACT)
    ideal = np.abs(plain(O.ROUNDING["bf16"]) - exact).max()
    t = torch.from_numpy(tok).cuda()
    first = {}
    for n in (300, 230, 129, 8, 1, 300, 230, 129, 8, 1, 264):
        h = torch.full((n, cfg.d_model), 7.0, device="cuda")
        m.armt_forward_full_attention(t[:n].contiguous(), h)
        torch.cuda.synchronize()
        m.armt_sync_status()
        # 1.5: the measured factor of tests/test_gpu_parity.py
        assert np.abs(h.double().cpu().numpy() - exact[:n]).max() <= 1.5 * ideal, n
        assert torch.equal(first.setdefault(n, h), h)
    m.close()
