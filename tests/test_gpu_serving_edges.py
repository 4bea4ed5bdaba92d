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
        with np.errstate(invalid="ignore"):
            off = got - ref
        less = ref + np.sign(off) * np.maximum(np.abs(off) - lost, 0.0)  # what is left to the other terms
        less = np.where(np.isfinite(off), less, got)
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


# new rows for each kernel over a bf16 cache, then over an e4m3 one (4 heads a kv head)
BOTH = [("bf16", 64, 1), ("bf16", 128, 3), ("bf16", 128, 7), ("bf16", 64, 12), ("bf16", 128, 40), ("bf16", 64, 40)] + \
    [("e4m3", hd, n) for hd, n in ROWS if hd == 64 or n != 8]


def minus_infinity(s, b, positions):
    """Makes the scores of sequence b's keys at `positions` -inf, for queries of 1 in column 0 and 0 elsewhere."""
    pos = np.array(positions)
    page, slot = (torch.from_numpy(x).long().cuda() for x in (s.table[b, pos // s.page], pos % s.page))
    if s.type == B.CACHE_BF16:
        s.cache.k[page, :, slot, 0] = -math.inf
    else:                                                    # -1 times infinity
        s.cache.k.view(torch.uint8)[page, :, slot] = 0xB8
        s.cache.k_scale[page, :, slot] = 255


def first_column(s):
    q = torch.zeros(s.n_rows, 4 * s.hkv, s.hd, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    if s.type == B.CACHE_E4M3:
        q[..., 1:] = 0.5                                     # (0 times infinity would be NaN)
    return q


@pytest.mark.parametrize("kv", [150, 20000])
@pytest.mark.parametrize("type_,hd,new", BOTH)
def test_a_row_whose_scores_are_all_minus_infinity(type_, hd, new, kv):
    """0 / 0: NaN.  A row that attends to nothing, in the same call, stays zero, and other sequences are not touched."""
    s = Wide(type_, 1, hd, 16, [new, 1, new, new], [kv, 33, 90, 40], seed=3)
    s.table[2] = -1                                          # its pages are gone
    s.batch = s.make_batch()
    minus_infinity(s, 0, range(kv))
    minus_infinity(s, 3, range(40))
    s.k, s.v = s.k.copy(), s.v.copy()
    for b, n in ((0, kv), (3, 40)):
        for pos in range(n):
            s.k[s.table[b, pos // 16], :, pos % 16] = 0.0
            s.k[s.table[b, pos // 16], :, pos % 16, 0] = -math.inf
    q = first_column(s)
    out = s.attend(q)
    first, other, gone, last = out.split([new, 1, new, new])
    assert first.isnan().all() and last.isnan().all()
    assert (gone == 0).all() and not other.isnan().any()
    # the definition says the same (in the plain form's columns: the others of q times 0)
    p = q.clone()
    if type_ == "e4m3":
        p[..., 1:] = 0
        p[new] = q[new]
    s.check(p, out)


@pytest.mark.parametrize("kv", [200, 20000])
@pytest.mark.parametrize("type_,hd,new", BOTH)
def test_some_keys_at_minus_infinity_have_no_weight(type_, hd, new, kv):
    """The front of a context at -inf, alone in the first part of one that is split."""
    s = Wide(type_, 1, hd, 16, [new, 2], [kv, 70], seed=3)
    front = range(kv - new - 40)
    minus_infinity(s, 0, front)
    q = first_column(s)
    got = s.attend(q)
    assert not got.isnan().any()
    # the plain form with -1,000 in their place, which leaves them e^-100 and keeps the check's bound on scores
    if type_ == "bf16":
        s.refresh()
    for pos in front:
        at = s.table[0, pos // 16], slice(None), pos % 16
        s.k[at] = 0.0
        s.k[at + (0,)] = -1000.0
    s.check(q, got)
    # a weight of 0 does not keep NaN out, also where the key's part has no other weight
    page, slot = int(s.table[0, 1]), 3
    if type_ == "bf16":
        s.cache.v[page, :, slot, 5] = math.nan
    else:
        s.cache.v.view(torch.uint8)[page, :, slot, 5] = 0x7F
    out = s.attend(q)
    assert out[:new, :, 5].isnan().all()
    out[:new, :, 5] = got[:new, :, 5]
    assert torch.equal(out, got)


@pytest.mark.parametrize("type_,hd", [("bf16", 64), ("bf16", 128), ("e4m3", 64), ("e4m3", 128)])
def test_non_finite_values_of_many_short_items(type_, hd):
    """The many-row kernel, several items of one or two key tiles for each block, every other one with values that are not
    finite in keys that only some of its rows see: each item's rows get its own, whatever the items beside it have."""
    rng = np.random.default_rng(11)
    n_seqs = 900
    kv = [int(x) for x in rng.integers(20, 180, n_seqs)]
    new = [min(int(x), k) for x, k in zip(rng.integers(9, 34, n_seqs), kv)]
    s = Wide(type_, 1, hd, 16, new, kv, seed=11, max_new=33)
    for b in range(n_seqs):
        for _ in range(int(rng.integers(0, 3))):
            pos = int(rng.integers(kv[b] - new[b], kv[b]))
            page, slot, col = int(s.table[b, pos // 16]), pos % 16, int(rng.integers(hd))
            if type_ == "bf16":
                s.cache.v[page, 0, slot, col] = float(rng.choice([math.nan, math.inf, -math.inf]))
            else:
                s.cache.v.view(torch.uint8)[page, 0, slot, col] = 0x7F
    if type_ == "bf16":
        s.refresh()
    else:
        set_codes(s)
    q = s.queries(4)
    out = s.attend(q)
    s.check(q, out)
    assert out.isfinite().any() and not out.isfinite().all()
    assert torch.equal(out.view(torch.int16), s.attend(q).view(torch.int16))


@pytest.mark.parametrize("type_", ["bf16", "e4m3"])
@pytest.mark.parametrize("starts", [
    [0, 100, 4, 8, 12], [0, 3, 1, 9, 12], [-2, 3, 6, 9, 12], [0, 3, 6, 9, 13], [4, 8, 0, 4, 2],
    [9, 3, 100, 5, 8] + [8] * 70 + [10, 0, 2, 1, 12]])
def test_rows_are_written_and_read_wherever_the_attention_takes_them_from(type_, starts):
    """Starts that decrease or leave the rows: those sequences have no rows, all others keep theirs."""
    n = len(starts) - 1
    s = Setup(type_, 2, 64, 16, [3] * n, [30] * n, seed=5)
    s.row_start, s.n_rows, s.max_new = np.array(starts, np.int32), 12, 12
    s.batch = s.make_batch()
    k, v = (torch.from_numpy(s.rng.standard_normal((12, 2, 64)).astype(np.float32)).bfloat16().cuda() for _ in range(2))
    B.armt_cache_write_bf16(k, v, s.cache, s.batch)
    back = [torch.full((12, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    B.armt_cache_read_bf16(s.cache, s.batch, *back)
    torch.cuda.synchronize()
    placed = P.places(s.row_start, s.kv_len, s.table, 16, s.n_pages, 12, 12)
    rows = [p[0] for p in placed]
    assert set(rows)
    for i, x in enumerate((k, v)):
        want = x.double().cpu().numpy()
        if type_ == "e4m3":
            codes, sc = P.quantise(want)
            want = P.e4m3_decode(codes) * np.exp2(sc.astype(np.float64) - 127)[..., None]
        want[np.setdiff1d(np.arange(12), rows)] = 7.0
        assert np.array_equal(back[i].double().cpu().numpy(), want)
        pool = s.cache.k if i == 0 else s.cache.v
        for row, b, pos, page in placed:
            if type_ == "bf16" and rows.count(row) == 1 and page >= 0:
                assert np.array_equal(pool[page, :, pos % 16].double().cpu().numpy(), want[row])


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 5, 43, 64])
def test_one_workspace_serves_smaller_batches_and_both_types(hd, group):
    setups = {t: Setup(t, 1, hd, 16, [40], [90], seed=2) for t in ("bf16", "e4m3")}
    sizes = {t: [B.armt_paged_attention_workspace(s.cache, s.make_batch(max_new=m), group)
                 for m in (1, 2, 3, 4, 7, 8, 9, 16, 17, 32, 33, 40)] for t, s in setups.items()}
    assert sizes["bf16"] == sizes["e4m3"] == sorted(sizes["bf16"])
    # the number of sequences does not matter, fewer rows than max_new do
    s = setups["bf16"]
    two = B.PagedBatch(torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"),
                       s.batch.page_table.repeat(2, 1), n_rows=40, max_new=40)
    assert B.armt_paged_attention_workspace(s.cache, two, group) == sizes["bf16"][-1]
    two = B.PagedBatch(two.row_start, two.kv_len, two.page_table, n_rows=3, max_new=40)
    assert B.armt_paged_attention_workspace(s.cache, two, group) == sizes["bf16"][2]
    workspace = torch.full((sizes["bf16"][-1],), 255, dtype=torch.uint8, device="cuda")
    for t, s in setups.items():
        for new in ([1], [3], [40]):
            s.row_start = np.array([0] + new, np.int32)
            s.max_new = new[0]
            q = s.queries(group)
            out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
            B.armt_paged_attention_bf16(q, s.cache, s.make_batch(), out, workspace)
            s.check(q, out)


@pytest.mark.parametrize("vocab", [37, 5000, 140001])
def test_a_temperature_of_nan_gives_nan_and_the_other_rows_their_probabilities(vocab):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(3, vocab, generator=g, device="cuda")
    x[1, 5] = -math.inf
    want, got = torch.empty_like(x), torch.empty_like(x)
    B.armt_token_probs(x, want, torch.tensor([0.7, 1.0, 0.0], device="cuda"))
    B.armt_token_probs(x, got, torch.tensor([0.7, math.nan, 0.0], device="cuda"))
    assert got[1].isnan().all() and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    assert not want.isnan().any()


# ------------------------------------------- paths that other tests leave out --

@pytest.mark.parametrize("kv", [100, 9000])
@pytest.mark.parametrize("hd,new", ROWS)
def test_nan_codes_that_are_seen(hd, new, kv):
    """NaN codes of an e4m3 cache, in values and keys of new rows: rows that see them get NaN, the others nothing of them."""
    s = Setup("e4m3", 1, hd, 16, [new, 1], [kv, 40], seed=6)
    codes = [x.view(torch.uint8).cpu().numpy() for x in (s.cache.k, s.cache.v)]

    def put(pool, pos, col):
        codes[pool][int(s.table[0, pos // 16]), 0, pos % 16, col] = 0x7F
    put(1, kv - 1, 5)                                        # seen by the last row alone
    put(1, kv - 1 - new // 2, 7)
    put(1, kv - new, 9)                                      # by all of them
    set_codes(s, k=codes[0], v=codes[1])
    q = s.queries(4)
    out = s.attend(q)
    s.check(q, out)
    assert out[new - 1, :, 5].isnan().all() and out[:new, :, 9].isnan().all() and out[new].isfinite().all()
    put(0, kv - 1, 3)                                        # the last row all NaN
    set_codes(s, k=codes[0])
    out = s.attend(q)
    s.check(q, out)
    assert out[new - 1].isnan().all()
    # and as the write makes them, of NaN and infinities
    k, v = (torch.randn(s.n_rows, 1, hd, generator=torch.Generator().manual_seed(i)).bfloat16().cuda() for i in range(2))
    v[0, 0, 1], v[new - 1, 0, 2], v[new - 1, 0, 3] = math.inf, -math.inf, math.nan
    B.armt_cache_write_bf16(k, v, s.cache, s.batch)
    set_codes(s)
    out = s.attend(q)
    s.check(q, out)
    assert out[:new, :, 1].isnan().all() and out[new - 1, :, 2].isnan().all() and out[new].isfinite().all()


@pytest.mark.parametrize("type_,hd,new", BOTH)
def test_more_sequences_than_a_warp_has_lanes(type_, hd, new):
    """The plan's sums over hundreds of sequences, each kernel; every third without rows, some with one."""
    rng = np.random.default_rng(5)
    kv = [int(x) for x in rng.integers(1, 120, 333)]
    rows = [0 if b % 3 == 1 else 1 if b % 5 == 0 else min(new, k) for b, k in enumerate(kv)]
    s = Setup(type_, 2, hd, 16, rows, kv, seed=8, max_new=new)
    q = s.queries(4)
    out = s.attend(q)
    s.check(q, out)
    assert torch.equal(out, s.attend(q))


@pytest.mark.parametrize("type_,hd,new", BOTH)
def test_hundreds_of_sequences_without_rows(type_, hd, new):
    """A few active sequences among idle ones, in front, between and behind; and the same ones by themselves."""
    n, active = 700, {0: 300, 350: 41, 351: 2000, 698: 77}
    kv = [active.get(b, 50 if b % 2 else 0) for b in range(n)]
    rows = [min(new, kv[b]) if b in active else 0 for b in range(n)]
    s = Setup(type_, 1, hd, 16, rows, kv, seed=8, max_new=new)
    q = s.queries(4)
    out = s.attend(q)
    s.check(q, out)
    ids = sorted(active)
    alone = B.PagedBatch(*(torch.from_numpy(np.ascontiguousarray(x)).cuda() for x in (
        np.concatenate([[0], np.cumsum([rows[b] for b in ids])]).astype(np.int32), s.kv_len[ids], s.table[ids])),
        n_rows=s.n_rows, max_new=new)
    assert torch.equal(out, s.attend(q, batch=alone))


@pytest.mark.parametrize("scale", [30.0, 1e-30, 1e4])
@pytest.mark.parametrize("type_,hd,new", BOTH)
def test_extreme_softmax_scales(type_, hd, new, scale):
    s = Wide(type_, 1, hd, 32, [new, 1], [400, 90], seed=8)
    q = s.queries(4)
    s.check(q, s.attend(q, scale=scale), scale=scale)


# -------------------------------------------------------- with the model --

def test_a_continued_sequence_equals_the_whole_one_through_the_model():
    """The full-attention baseline's layers around the cache and the attention, fed a prompt's chunk, then drafted tokens,
    then single ones, for two packed sequences: the hidden states of armt_forward_full_attention over the whole sequences.

    Weight products are the library's; norms, rotary embedding and SwiGLU are written out here.  Against the definition in
    64 bits the error stays within 1.5 times that of ideal arithmetic with the same operands rounded to bf16, the factor
    that tests/test_gpu_parity.py measures; so do the baseline's own (with fp16 operands in its attention), and the two
    therefore differ by no more than the sum."""
    import dataclasses

    from oracle import armt_oracle as O
    from recurrent_memory_transformer_gb300 import inputs as I
    cfg = dataclasses.replace(I.ARMT_1B, n_layers=2, vocab=4096)
    W = I.make_weights(cfg, seed=61, norm_jitter=0.1)
    m = B.Model(cfg, B.device_weight_tensors(cfg, W))
    lens = [230, 130]
    tok = [np.random.default_rng(61 + b).integers(0, cfg.vocab, size=n).astype(np.int32) for b, n in enumerate(lens)]
    hq, hkv, hd, d = cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim, cfg.d_model
    wide = {k: torch.from_numpy(np.asarray(v, np.float32)).cuda() for k, v in W.items()}

    def norm(x, gain):
        x = x.double()
        return (x / (x.square().mean(-1, keepdim=True) + cfg.norm_eps).sqrt() * gain.double()).bfloat16()

    def product(x, w):
        out = torch.empty(1, x.shape[0], w.shape[0], dtype=torch.float32, device="cuda")
        B.armt_grouped_gemm_bf16(x.contiguous()[None], w.bfloat16().contiguous()[None], out)
        return out[0]

    def rope(x, pos):
        half = hd // 2
        angle = pos.double()[:, None, None] * (cfg.rope_base ** (-2.0 * torch.arange(half, device="cuda").double() / hd))
        a, b = x.double()[..., :half], x.double()[..., half:]
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1).bfloat16()

    pages = torch.randperm(40, generator=torch.Generator().manual_seed(1)).int().cuda()[:36].view(2, 18)[:, :15].contiguous()
    caches = [B.KvCache.allocate(40, 16, hkv, hd) for _ in range(cfg.n_layers)]
    got = [torch.empty(n, d, device="cuda") for n in lens]
    done = [0, 0]
    steps = [(180, 100), (5, 3), (1, 5), (4, 0)] + [(1, 1)] * 40
    for step in steps:
        new = [min(n, total - at) for n, total, at in zip(step, lens, done)]
        if not sum(new):
            continue
        done = [at + n for at, n in zip(done, new)]
        batch = B.PagedBatch(torch.tensor([0, new[0], sum(new)], dtype=torch.int32, device="cuda"),
                             torch.tensor(done, dtype=torch.int32, device="cuda"), pages, sum(new), max(new))
        workspace = B.paged_attention_workspace(caches[0], batch, hq)
        pos = torch.cat([torch.arange(at - n, at, device="cuda") for n, at in zip(new, done)])
        ids = torch.from_numpy(np.concatenate([t[at - n:at] for t, n, at in zip(tok, new, done)])).long().cuda()
        x = wide["embed"][ids]
        for l, cache in enumerate(caches):
            n1 = norm(x, wide["norm1"][l])
            q, k, v = (product(n1, wide[w][l]).unflatten(1, (-1, hd)) for w in ("wq", "wk", "wv"))
            B.armt_cache_write_bf16(rope(k, pos), v.bfloat16(), cache, batch)
            out = torch.empty(sum(new), hq, hd, dtype=torch.bfloat16, device="cuda")
            B.armt_paged_attention_bf16(rope(q, pos), cache, batch, out, workspace)
            x = x + product(out.flatten(1), wide["wo"][l])
            n2 = norm(x, wide["norm2"][l])
            gate, up = product(n2, wide["w_gate"][l]), product(n2, wide["w_up"][l])
            x = x + product((torch.nn.functional.silu(gate.double()) * up.double()).bfloat16(), wide["w_down"][l])
        y = x.double()
        y = y / (y.square().mean(-1, keepdim=True) + cfg.norm_eps).sqrt() * wide["norm_f"].double()
        for b, part in enumerate(y.float().split(new)):
            got[b][done[b] - new[b]:done[b]] = part
    assert done[0] >= 229 and done[1] == lens[1]
    B.armt_block_sync_status()

    def plain(rounding, t):
        W64 = O.widen_weights(W)
        x = W64["embed"][t]
        for l in range(cfg.n_layers):
            x = O.llama_block(x, cfg, W64, l, rounding)
        return O.rmsnorm(x, W64["norm_f"], cfg.norm_eps)
    for b, n in enumerate(done):
        h = torch.empty((n, d), dtype=torch.float32, device="cuda")
        m.armt_forward_full_attention(torch.from_numpy(tok[b][:n]).cuda(), h)
        m.armt_sync_status()
        exact = plain(O.EXACT, tok[b][:n])
        ideal = np.abs(plain(O.OperandRounding(O.round_bf16, O.round_bf16), tok[b][:n]) - exact).max()
        half = np.abs(plain(O.ROUNDING["bf16"], tok[b][:n]) - exact).max()
        here = got[b][:n].double().cpu().numpy()
        assert np.abs(here - exact).max() <= 1.5 * ideal, (np.abs(here - exact).max(), ideal)
        assert np.abs(here - h.double().cpu().numpy()).max() <= 1.5 * (ideal + half)
        assert (here * exact).sum() / np.linalg.norm(here) / np.linalg.norm(exact) >= 0.999
    m.close()


@pytest.mark.parametrize("type_,hd,new", BOTH)
def test_long_contexts_without_pages(type_, hd, new):
    """Tables of 65,536 pages that are all missing give zeros, beside a sequence whose only page, thousands of missing ones
    in, has scores of -inf: NaN."""
    s = Setup(type_, 1, hd, 16, [new] * 3, [40] * 3, seed=4, width=65536)
    table = torch.full((3, 65536), -1, dtype=torch.int32, device="cuda")
    table[1, 60000] = int(s.table[0, 0])
    s.table[1, 0] = s.table[0, 0]
    minus_infinity(s, 1, range(16))
    lens = torch.full((3,), 65536 * 16, dtype=torch.int32, device="cuda")
    q = first_column(s)
    out = s.attend(q, batch=B.PagedBatch(s.batch.row_start, lens, table, s.n_rows, new))
    B.armt_block_sync_status()
    assert (out[:new] == 0).all() and out[new:2 * new].isnan().all() and (out[2 * new:] == 0).all()
