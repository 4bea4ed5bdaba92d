// Attention of a batch's new rows over the paged cache.
//
//   out_i = sum_j w_ij v_j / sum_j w_ij,  w_ij = 2^(c q_i . k_j),  c = scale * log2(e)
//
// over the visible keys j, evaluated in one pass with a running maximum
// (how, is said at the kernels).  Query heads of one kv head share its
// keys, so a query tile's rows are (token, head of the group) pairs: row =
// token * group + head.
#include <algorithm>
#include <type_traits>

#include "paged_attn.cuh"

namespace armt {
namespace {

// ------------------------------------------------------ few query rows --
//
// One token a sequence, or a few drafted ones: up to 64 rows against
// thousands of keys, so the kernel streams the cache once and HBM bounds it.
// What the streams need is bytes in flight (about 6.7 TB/s x 0.8 us = 35 KB
// per SM, several times that to ride out the spread of latencies) and few
// instructions beside the products: a producer warp walks the page table (32
// page ids a load) and has TMA fetch tiles of 64 keys, K and V, 8 to 32 KB, a
// box for each run of keys in one page, into STAGES buffers; four consumer
// warps wait for a buffer, use it and hand it back, without waiting for one
// another; two or three blocks share an SM.
//
// The products run on mma.sync (m16n8k16): a 128-row tcgen05 tile would be
// mostly padding, and the tensor rate is not what bounds here.  Up to 16 rows
// they are turned round (turned_kernel): keys and value columns take the 16-row
// side, the rows one or two 8-column tiles, and each of the four warps has 16
// of a tile's 64 keys, so that a cached element is read and converted once.
// For 17 to 32 rows, 64 with head_dim 64 (rows_kernel), the rows fill two or
// four 16-row tiles; two warps of different rows, or four, read the same keys.  (21 rows, bf16: 70 us
// so, 80 with three 8-column tiles, whose sums spill.)
//
// Work is dealt out in tiles, not in sequences: every block takes an equal,
// contiguous range of the list of (sequence, kv head, query tile, key tile),
// so ragged batches balance by construction; a sequence whose tiles fall to
// several blocks leaves parts (fp32 sums with their references) that the joining
// kernel adds in block order.
//
// What is held in fewer than 32 bits: the weights, as operands of the second
// product, which takes 16-bit ones: rounded to V's bf16 (2^-8 of each), over codes
// to fp16 (2^-11).  Their sum is taken in fp32 before that.  Against 64 bits the
// outputs are off by 0.0021 to 0.0023 (bf16) and 0.0017 (codes) of their size, of
// which the rounding of the output to bf16 alone is 0.0017.
//
// e4m3 caches: codes go to fp16 by one conversion instruction for two values
// (exact), the products run on fp16 with q scaled by a power of two per row
// (exact down to 2^-28 of the row's largest), the key's scale multiplies the
// score.  The value's scale 2^e joins the weight, and the running maximum m
// is taken of score + e, so the fp16 weights stay in range whatever the scales:
// the largest is at least 2^7 and at most 2^15, and fp16's subnormals are 2^-24
// apart (a weight is off by 2^-11 of itself, or 2^-32 of the largest).
//
// The weights of the sum l go without e.  While every e is within 60 of 0, one
// exponential 2^(score - m) serves both: the sum's terms are at most 2^75, the
// largest at least 2^-53, and what ends at 2^-126 matters to neither.  From the
// first tile with an e beyond that (bf16 rows past 2^69, or all below 2^-51) a
// warp's item is wide: l then has a maximum u of the scores alone and an
// exponential of its own, the weight is 2^(score - m + e), and the output is
// sum / l * 2^(m - u).  The first exponents beyond are found where the reference
// is about to move, and send the tile to the wide form, so that the others pay a
// comparison and some registers (16 sequences to 8K: 59 us with 12 rows, 83 with
// 28, 88 with 64 of head_dim 64; one reference for all, wrong beyond: 56, 85, 86;
// two exponentials for all: 62, 91, 104).

constexpr int kKeys = 64;      // keys of a tile
constexpr int kThreads = 128;  // of the four consumer warps
// What an item costs beside its tiles, in keys, for dealing out the work (64 x
// 1 e4m3: 269 us with 64 keys, 181 with 192, 174 with 320, 175 with 512).
constexpr int kFixedKeys = 5 * kKeys;

// NB: turned products, 8 NB rows; 0: WM 16-row tiles.
template <int HD, int TYPE, int NB, int WM = 0>
struct RowsCfg {
  static constexpr bool B16 = TYPE == ARMT_CACHE_BF16;
  static constexpr int ROW = B16 ? HD * 2 : HD;       // bytes of a cached row
  static constexpr int LINE = ROW < 128 ? ROW : 128;  // bytes of a row in shared memory, swizzled over LINE
  static constexpr int ATOMS = ROW / LINE;            // a longer row is this many such lines, kKeys lines apart
  static constexpr int POOL = kKeys * ROW;
  static constexpr int SCALES = B16 ? 0 : 2 * kKeys;
  static constexpr int STAGE = (2 * POOL + SCALES + 1023) / 1024 * 1024;
  // resident on an SM: registers, mostly (64 rows over codes: 88 us, 100 with three blocks, whose sums spill)
  static constexpr int BLOCKS = (HD == 64 && (B16 || WM != 4)) || (NB == 1 && !B16) ? 3 : 2;
  static constexpr int JOIN = 2 * 32 * 32 * 4;  // two warps' pieces of 32 values a lane
  static constexpr int QUERIES = NB * HD * 16;  // turned: the queries' fragments
  // as many buffers, up to 6, as those blocks find room for beside a KB that
  // each block costs, its static shared memory and a KB of alignment
  static constexpr int ROOM = 233472 / BLOCKS - 1024 - (12 * HD + 1024) - 1024 - JOIN - QUERIES;
  static constexpr int STAGES = ROOM / STAGE < 6 ? ROOM / STAGE : 6;
  static_assert(STAGES >= 2, "a buffer to fill beside the one in use");
  static constexpr int SMEM = 1024 + STAGES * STAGE + JOIN + QUERIES;
};

// Set by a bounded wait that gave up; the joining kernel passes it on.
__device__ int g_paged_err;

// Barrier of the consumer warps.
__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// Barrier of the consumer warps that also says whether any thread had `mine`.
__device__ __forceinline__ bool consumers_any(bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)mine)
      : "memory");
  return any != 0;
}

template <int TYPE>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (TYPE == ARMT_CACHE_BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Whether a value's scale byte is beyond what one reference serves; and the
// exponent of a byte in the weights of a wide item: -inf for a scale of zero,
// +inf for infinity.
__device__ __forceinline__ bool wide_scale(uint32_t byte) { return byte - 67u > 120u; }
__device__ __forceinline__ float scale_exponent(uint32_t byte) {
  return byte == 0u ? -INFINITY : byte == 255u ? INFINITY : (float)((int)byte - 127);
}

// What a row's sum of products in reference m is multiplied by, one after the
// other, for its output: 1 / l, l in reference u (see weight_share), and
// 2^(m - u) in two halves (it may be 2^140).
struct RowFactors {
  float first, second;
};
__device__ __forceinline__ RowFactors row_factors(float l, float m, float u) {
  // weight_share(l, m) with the hardware's reciprocal (2^-22 off), which spills
  // less: 12 rows over codes 59 us for 61, 28 rows 83 for 86
  const float inv = l == 0.f ? (m == -INFINITY ? 0.f : NAN) : __fdividef(1.f, l);
  const float half = m == u ? 1.f : fast_exp2(0.5f * (m - u));
  return RowFactors{inv * half, half};
}

// Two e4m3 codes (low 16 bits) -> two fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

// Barriers and buffers of a block.
template <typename C>
struct RowsShared {
  PlanScratch scratch;
  PlanRange range;
  uint64_t full[C::STAGES], empty[C::STAGES];
  uint32_t with_page[C::STAGES];  // 4 bits: which 16-key groups of the tile have a page
};

template <typename C>
__device__ __forceinline__ void init_barriers(RowsShared<C>& sh) {
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 4);
    }
    fence_barrier_init();
    fence_proxy_async_smem();
  }
}

// The producer warp: the range's tiles, one after another, into the buffers.
template <typename C>
__device__ __forceinline__ void produce(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const PagedArgs& a,
                                        const PagedView& p, const PlanRange& range, RowsShared<C>& sh, uint8_t* smem) {
  constexpr bool B16 = C::B16;
  const int lane = threadIdx.x & 31;
  int* err = &g_paged_err;
  PlanCursor at = range.first;
  const int run = min(1 << p.page_shift, kKeys);  // keys of a tile that share a page
  const uint32_t run_bits = (1u << (run / 16)) - 1u;
  int ids = -1;        // page of the run that starts at key ids_at + run * lane
  int ids_at = -1, ids_b = -1;
  int stage = 0, issued = 0;
  uint32_t phase = 1;  // the buffers start out empty
  // the tiles of an item, then on to the next
  for (bool more = true; more; more = plan_next_item(a.plan, p, range, at)) {
    const int count = plan_here(range, at);
    bool ok = true;
    for (int j0 = 0; ok && j0 < count; ++j0) {
      const int k0 = (at.tile + j0) * kKeys;
      if (at.b != ids_b || k0 < ids_at || k0 + kKeys - ids_at > 32 * run) {
        ids_b = at.b;
        ids_at = k0;
        const long long key = (long long)k0 + run * lane;
        ids = key < at.kv ? paged_page(p, at.b, key) : -1;
      }
      ok = issued != a.wp.stall_after && mbar_wait_bounded(&sh.empty[stage], phase, err, DEV_TIMEOUT_EMPTY, a.wp.limit_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      // lane j has the copies of run j
      const int page = __shfl_sync(0xffffffffu, ids, (k0 - ids_at) / run + lane & 31);
      const bool mine = lane < kKeys / run && page >= 0;
      const uint32_t have = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) {
        uint32_t groups = 0;
        for (int j = 0; j < kKeys / run; ++j) groups |= (have >> j & 1u) * (run_bits << (j * run / 16));
        sh.with_page[stage] = groups;
        mbar_arrive_expect_tx(&sh.full[stage], (uint32_t)(__popc(have) * 2 * run * (C::ROW + (B16 ? 0 : 1))));
      }
      __syncwarp();
      if (mine) {
        uint8_t* sk = smem + stage * C::STAGE;
        const int key = lane * run, slot = (k0 + key) & ((1 << p.page_shift) - 1), head = page * p.hkv + at.head;
#pragma unroll
        for (int t = 0; t < C::ATOMS; ++t) {
          const int dst = t * kKeys * C::LINE + key * C::LINE;
          tma_load_3d(sk + dst, &tm_k, t * 64, slot, head, &sh.full[stage]);
          tma_load_3d(sk + C::POOL + dst, &tm_v, t * 64, slot, head, &sh.full[stage]);
        }
        if constexpr (!B16) {
          const long long row = paged_row(p, page, at.head, slot);
          bulk_load(sk + 2 * C::POOL + key, p.k_scale + row, run, &sh.full[stage]);
          bulk_load(sk + 2 * C::POOL + kKeys + key, p.v_scale + row, run, &sh.full[stage]);
        }
      }
      ++issued;
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) break;
  }
  // every copy has landed before the block lets go of its shared memory
  if (lane == 0)
    for (int k = max(0, issued - C::STAGES); k < issued; ++k)
      mbar_wait_drain(&sh.full[k % C::STAGES], (uint32_t)(k / C::STAGES & 1));
}

template <int HD, int TYPE, int WM>
__global__ void __launch_bounds__(kThreads + 32, RowsCfg<HD, TYPE, 0, WM>::BLOCKS)
    rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedArgs a,
                const PagedView p) {
  using C = RowsCfg<HD, TYPE, 0, WM>;
  constexpr int WN = 4 / WM;             // warps that share rows and split keys
  constexpr int KPW = kKeys / WN;        // keys of a tile for one warp
  constexpr int R = 16 * WM;             // rows of a query tile
  constexpr int NT = HD / 8;             // 8-column tiles of the output
  constexpr float kNominal = TYPE == ARMT_CACHE_BF16 ? 0.f : 7.f, kRaise = kNominal + 8.f;
  constexpr bool B16 = TYPE == ARMT_CACHE_BF16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ Poison bad[HD];
  __shared__ RowsShared<C> sh;
  __shared__ float sum_ref[B16 ? 1 : 4][16];  // wide items: u of each warp's rows
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % WM, wn = warp / WM;
  const int r = lane >> 2, c = lane & 3;
  const uint32_t sbase = smem_u32(smem);
  float* join = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
  int* err = &g_paged_err;

  for (int i = tid; i < HD; i += kThreads + 32) bad[i] = Poison{0x7fffffff, 0x7fffffff, 0x7fffffff};
  init_barriers<C>(sh);
  // the joining kernel may be brought in; it waits for this one's end before
  // it reads anything that this one writes
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  plan_and_keep(a, p, sh.scratch, sh.range);  // the block has met: barriers and notes are set up
  const PlanRange& range = sh.range;
  if (range.empty) return;

  if (warp == 4) {
    produce<C>(tm_k, tm_v, a, p, range, sh, smem);
    return;
  }

  // ---- consumers
  PlanCursor at = range.first;
  uint32_t qf[HD / 16][4];
  float o[NT][4];
  float m[2], l[2];
  float row_scale[2];
  int visible[2];  // keys this thread's two rows see
  int seen_min = 0, seen_max = 0;
  bool noted = false;  // this thread has written to `bad` for the query tile
  bool wide = false;   // this warp's sums have two references (the same for all its lanes)
  int paged_from = 0;  // the first key of the item, in this block's part of it, that has a page

  // reads the rows of the query tile at `at`, and starts its sums
  auto start_item = [&]() {
    const int rows = at.n * a.plan.group;
    noted = wide = false;
    int qrow[2];
    bool valid[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = at.qt * R + 16 * wm + r + 8 * h;
      qrow[h] = row;
      valid[h] = row < rows;
      const int tok = row / a.plan.group;
      visible[h] = valid[h] ? plan_visible(at, tok) : 0;
      m[h] = -INFINITY;
      l[h] = 0.f;
      row_scale[h] = a.scale_log2;
    }
    seen_min = plan_visible(at, at.qt * R / a.plan.group);
    seen_max = plan_visible(at, min(rows - 1, at.qt * R + R - 1) / a.plan.group);
#pragma unroll
    for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    if constexpr (B16) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = qrow[h] / a.plan.group, head = at.head * a.plan.group + qrow[h] % a.plan.group;
        const uint32_t* src =
            reinterpret_cast<const uint32_t*>(a.q + (long long)(at.row0 + tok) * a.q_stride + head * HD) + c;
#pragma unroll
        for (int s = 0; s < HD / 16; ++s) {
          qf[s][h] = valid[h] ? __ldg(src + 8 * s) : 0u;
          qf[s][2 + h] = valid[h] ? __ldg(src + 8 * s + 4) : 0u;
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int tok = qrow[h] / a.plan.group, head = at.head * a.plan.group + qrow[h] % a.plan.group;
        const uint2* src = reinterpret_cast<const uint2*>(a.q + (long long)(at.row0 + tok) * a.q_stride + head * HD);
        float top = 0.f;
        uint2 w[HD / 16];
#pragma unroll
        for (int s = 0; s < HD / 16; ++s) {  // step s of block s / 4: elements 64 (s / 4) + 16 c + 4 (s % 4) + 0..3
          w[s] = valid[h] ? __ldg(src + 16 * (s >> 2) + 4 * c + (s & 3)) : make_uint2(0u, 0u);
          const uint32_t x[2] = {w[s].x, w[s].y};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            top = fmaxf(top, fabsf(__uint_as_float(x[i] << 16)));
            top = fmaxf(top, fabsf(__uint_as_float(x[i] & 0xffff0000u)));
          }
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // q * 2^up has its largest element in [2^14, 2^15)
        const int up = min(100, 14 - ((int)(__float_as_uint(top) >> 23) - 127));
        const float f = __uint_as_float((uint32_t)(127 + max(up, -126)) << 23);
        row_scale[h] = a.scale_log2 / f;
#pragma unroll
        for (int s = 0; s < HD / 16; ++s) {
          qf[s][h] = pack_f16x2(__uint_as_float(w[s].x << 16) * f, __uint_as_float(w[s].x & 0xffff0000u) * f);
          qf[s][2 + h] = pack_f16x2(__uint_as_float(w[s].y << 16) * f, __uint_as_float(w[s].y & 0xffff0000u) * f);
        }
      }
    }
  };

  // The tile in `stage`: scores, weights, and their product with the values.
  // `mask`: not every row sees all of it, or some of it has no page; what lies
  // in such slots is taken out before it can touch a sum.  Not in the wide form
  // and an exponent that wants it: false, and nothing done.
  auto add_tile = [&](int stage, int k0, auto mask, auto wide_form) {
    const uint32_t sk = sbase + stage * C::STAGE, sv = sk + C::POOL;
    const int kw = wn * KPW;  // this warp's first key of the tile
    const uint32_t ok = mask() ? sh.with_page[stage] : 15u;
    // byte of a row's 16-byte piece
    auto piece_at = [&](int row, int piece) {
      if constexpr (C::LINE == 64) return row * 64 + ((piece ^ (row >> 1 & 3)) << 4);
      return (piece >> 3) * (kKeys * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
    };
    // the key (of 8) behind score column 2c + j, and of the value row read for
    // it: with 2c and 2c ^ 5 the reads below meet no bank twice (e4m3); bf16
    // fragments are fixed by ldmatrix
    auto key_of = [&](int col) { return B16 ? col : (col & 1 ? (col & 6) ^ 5 : col); };
    float s[KPW / 8][4];
#pragma unroll
    for (int t = 0; t < KPW / 8; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
    if constexpr (B16) {
      const int lrow = lane & 7, lmat = lane >> 3;
#pragma unroll
      for (int ks = 0; ks < HD / 16; ++ks) {
#pragma unroll
        for (int t = 0; t < KPW / 8; t += 2) {
          const int row = kw + 8 * (t + (lmat >> 1)) + lrow, piece = 2 * ks + (lmat & 1);
          uint32_t b[4];
          ldsm4(b, sk + piece_at(row, piece));
          mma16816<TYPE>(s[t], qf[ks], b[0], b[1]);
          mma16816<TYPE>(s[t + 1], qf[ks], b[2], b[3]);
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < KPW / 8; ++t) {
        const int row = kw + 8 * t + key_of(r);
#pragma unroll
        for (int blk = 0; blk < HD / 64; ++blk) {
          const uint4 w = lds128(sk + piece_at(row, 4 * blk + c));
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma16816<TYPE>(s[t], qf[4 * blk + i], e4m3x2_to_f16x2(ww[i]), e4m3x2_to_f16x2(ww[i] >> 16));
        }
      }
    }
    // to log2 units, masked
    [[maybe_unused]] float ve[KPW / 8][2];  // e4m3: the value scale (wide: its exponent) of this thread's keys
    [[maybe_unused]] bool beyond = false;   // one of them wants the wide form
    bool moves = wide_form();  // a row's reference has to move (see turned_kernel)
    float mx[2] = {-INFINITY, -INFINITY};
    [[maybe_unused]] float uref[2];
#pragma unroll
    for (int t = 0; t < KPW / 8; ++t) {
      [[maybe_unused]] float kf[2] = {1.f, 1.f}, ev[2] = {0.f, 0.f};
      if constexpr (!B16) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t at_key = sk + 2 * C::POOL + kw + 8 * t + key_of(2 * c + i);
          uint32_t kbyte = lds_u8(at_key), vbyte = lds_u8(at_key + kKeys);
          if (mask() && (k0 + kw + 8 * t + key_of(2 * c + i) >= seen_max || !(ok >> ((kw + 8 * t) >> 4) & 1u)))
            kbyte = vbyte = 127;  // seen by no row: may be anything
          kf[i] = scale_of(kbyte);
          ve[t][i] = wide_form() ? scale_exponent(vbyte) : scale_of(vbyte);
          ev[i] = (float)((int)vbyte - 127);
          beyond |= !wide_form() && wide_scale(vbyte);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = i >> 1, j = i & 1;
        float x = s[t][i] * row_scale[h];
        if constexpr (!B16) x *= kf[j];
        if (mask()) {
          const int key = kw + 8 * t + key_of(2 * c + j);
          if (k0 + key >= visible[h] || !(ok >> (key >> 4) & 1u)) x = -INFINITY;
        }
        s[t][i] = x;
        mx[h] = fmaxf(mx[h], B16 ? x : x + ev[j]);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) moves |= mx[h] > m[h] + kRaise;
    if (__any_sync(0xffffffffu, moves || beyond)) {
      if (!B16 && !wide_form() && __any_sync(0xffffffffu, beyond)) return false;
      float corr[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        const float next = fmaxf(m[h], mx[h] - kNominal), ref = next == -INFINITY ? 0.f : next;
        corr[h] = m[h] == next ? 1.f : fast_exp2(m[h] - ref);
        if constexpr (wide_form()) {
          const float from = wide ? sum_ref[warp][r + 8 * h] : m[h];
          float up = from;
#pragma unroll
          for (int t = 0; t < KPW / 8; ++t) up = fmaxf(up, fmaxf(s[t][2 * h], s[t][2 * h + 1]));
          up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 1));
          up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, 2));
          l[h] *= from == up ? 1.f : fast_exp2(from - up);
          uref[h] = up == -INFINITY ? 0.f : up;
          __syncwarp();
          if (c == 0) sum_ref[warp][r + 8 * h] = up;
        } else {
          l[h] *= corr[h];
        }
        m[h] = next;
      }
      if constexpr (wide_form()) {
        wide = true;
        __syncwarp();
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        o[t][0] *= corr[0];
        o[t][1] *= corr[0];
        o[t][2] *= corr[1];
        o[t][3] *= corr[1];
      }
    }
    const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int t = 0; t < KPW / 8; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (wide_form()) {
          const float x = s[t][i];
          l[i >> 1] += fast_exp2(x - uref[i >> 1]);
          s[t][i] = fast_exp2(x - ref[i >> 1] + ve[t][i & 1]);
          if (x == -INFINITY) s[t][i] = 0.f;  // a masked slot's scale byte may say infinity
        } else {
          const float w = fast_exp2(s[t][i] - ref[i >> 1]);
          l[i >> 1] += w;
          s[t][i] = w;
          if constexpr (!B16) s[t][i] = w * ve[t][i & 1];
        }
      }
    }
    // O += W V over this warp's keys, 16 at a time
#pragma unroll
    for (int kk = 0; kk < KPW / 16; ++kk) {
      uint32_t w[4];
      w[0] = pack2<typename std::conditional<B16, bf16, f16>::type>(s[2 * kk][0], s[2 * kk][1]);
      w[1] = pack2<typename std::conditional<B16, bf16, f16>::type>(s[2 * kk][2], s[2 * kk][3]);
      w[2] = pack2<typename std::conditional<B16, bf16, f16>::type>(s[2 * kk + 1][0], s[2 * kk + 1][1]);
      w[3] = pack2<typename std::conditional<B16, bf16, f16>::type>(s[2 * kk + 1][2], s[2 * kk + 1][3]);
      // x holds 16-bit values of keys kw + 16 kk + key[0] and key[1] in column
      // col.  Slots that no row sees are cleared; what is not finite among the
      // keys that only some rows see is noted and cleared.
      auto clean = [&](uint32_t& x, int key0, int key1, int col) {
        constexpr uint32_t E = B16 ? 0x7f80u : 0x7c00u;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int key = kw + 16 * kk + (half ? key1 : key0);
          const uint32_t y = x >> (16 * half) & 0xffffu;
          const bool unseen = k0 + key >= seen_max || !(ok >> (key >> 4) & 1u);
          if (!unseen && ((y & E) != E || k0 + kKeys <= seen_min)) continue;
          if (!unseen) {
            int* slot = (y & ~(E | 0x8000u)) != 0 ? &bad[col].nan : (y & 0x8000u) ? &bad[col].neg : &bad[col].pos;
            atomicMin(slot, k0 + key);
            noted = true;
          }
          x &= half ? 0x0000ffffu : 0xffff0000u;
        }
      };
      if constexpr (B16) {
        const int lrow = lane & 7, lmat = lane >> 3;
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          const int row = kw + 16 * kk + 8 * (lmat & 1) + lrow, piece = t + (lmat >> 1);
          uint32_t b[4];
          ldsm4t(b, sv + piece_at(row, piece));
          if (mask()) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              clean(b[i], 2 * c + 8 * (i & 1), 2 * c + 8 * (i & 1) + 1, 8 * (t + (i >> 1)) + r);
          }
          mma16816<TYPE>(o[t], w, b[0], b[1]);
          mma16816<TYPE>(o[t + 1], w, b[2], b[3]);
        }
      } else {
        // lane (r, c) takes columns NT r .. NT r + NT - 1 of the keys of score columns 2c, 2c + 1 of both 8s
        uint32_t x[4][NT / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = kw + 16 * kk + key_of(2 * c + (i & 1)) + 8 * (i >> 1);
          if constexpr (HD == 128) {
            const uint4 v = lds128(sv + piece_at(row, r));
            x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
          } else {
            const uint2 v = lds64(sv + piece_at(row, r >> 1) + 8 * (r & 1));
            x[i][0] = v.x, x[i][1] = v.y;
          }
        }
#pragma unroll
        for (int q4 = 0; q4 < NT / 4; ++q4) {
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // bytes 2 half, 2 half + 1 of the two keys, paired by column
            const uint32_t sel = half ? 0x7362u : 0x5140u;
            const uint32_t lo = __byte_perm(x[0][q4], x[1][q4], sel), hi = __byte_perm(x[2][q4], x[3][q4], sel);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int t = 4 * q4 + 2 * half + i;
              uint32_t b0 = e4m3x2_to_f16x2(lo >> (16 * i)), b1 = e4m3x2_to_f16x2(hi >> (16 * i));
              if (mask()) {
                const int k0c = key_of(2 * c), k1c = key_of(2 * c + 1);
                clean(b0, k0c, k1c, NT * r + t);
                clean(b1, k0c + 8, k1c + 8, NT * r + t);
              }
              mma16816<TYPE>(o[t], w, b0, b1);
            }
          }
        }
      }
    }
    return true;
  };

  // column of o[t][0] (and o[t][2]); o[t][1] is `next` further
  auto column = [&](int t) { return B16 ? 8 * t + 2 * c : 2 * NT * c + t; };
  constexpr int kNext = B16 ? 1 : NT;

  // joins the warps' sums and writes the query tile's rows, or its partial sums
  auto finish_item = [&](bool whole, int slot) {
    [[maybe_unused]] float u[2];  // codes: the reference of l
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      m[h] = seen_reference(m[h], paged_from < visible[h]);
      if constexpr (!B16) u[h] = wide ? sum_ref[warp][r + 8 * h] : m[h];
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
    // the upper half of the warps that share rows hands its sums to the lower half
#pragma unroll
    for (int half = WN / 2; half > 0; half /= 2) {
      const bool gives = wn >= half && wn < 2 * half, takes = wn < half;
      const int box = (wn % half) * WM + wm;  // at most two boxes
      float f_mine[2] = {1.f, 1.f}, f_other[2] = {1.f, 1.f};
      consumers_sync();
      if (gives) {
        *reinterpret_cast<float4*>(join + (box * 32 + lane) * 4) = make_float4(m[0], m[1], l[0], l[1]);
        if constexpr (!B16) *reinterpret_cast<float2*>(join + 256 + (box * 32 + lane) * 2) = make_float2(u[0], u[1]);
      }
      consumers_sync();
      if (takes) {
        const float4 y = *reinterpret_cast<const float4*>(join + (box * 32 + lane) * 4);
        const float om[2] = {y.x, y.y}, ol[2] = {y.z, y.w};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float top = fmaxf(m[h], om[h]), ref = top == -INFINITY ? 0.f : top;
          f_mine[h] = fast_exp2(m[h] - ref);
          f_other[h] = fast_exp2(om[h] - ref);
          if constexpr (B16) {
            l[h] = l[h] * f_mine[h] + ol[h] * f_other[h];
          } else {
            const float ou = join[256 + (box * 32 + lane) * 2 + h];
            const float up = fmaxf(u[h], ou), uref = up == -INFINITY ? 0.f : up;
            l[h] = l[h] * fast_exp2(u[h] - uref) + ol[h] * fast_exp2(ou - uref);
            u[h] = up;
          }
          m[h] = top;
        }
      }
#pragma unroll
      for (int t0 = 0; t0 < NT; t0 += 8) {  // 32 values a lane at a time
        consumers_sync();
        if (gives) {
#pragma unroll
          for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) join[(box * 32 + 4 * t + i) * 32 + lane] = o[t0 + t][i];
        }
        consumers_sync();
        if (takes) {
#pragma unroll
          for (int t = 0; t < 8; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              o[t0 + t][i] = o[t0 + t][i] * f_mine[i >> 1] + join[(box * 32 + 4 * t + i) * 32 + lane] * f_other[i >> 1];
        }
      }
    }
    const bool poisoned = consumers_any(noted);  // every warp has noted its non-finite values
    if (wn == 0) {
      if (poisoned) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            o[t][i] += poison_of(bad[column(t) + (i & 1) * kNext], visible[i >> 1]);
      }
      const int rows = at.n * a.plan.group;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int lr = 16 * wm + r + 8 * h, row = at.qt * R + lr;
        if (row >= rows) continue;
        if (whole) {
          const int tok = row / a.plan.group, head = at.head * a.plan.group + row % a.plan.group;
          bf16* dst = a.out + (long long)(at.row0 + tok) * a.out_stride + head * HD;
          if constexpr (B16) {
            const float inv = weight_share(l[h], m[h]);
#pragma unroll
            for (int t = 0; t < NT; ++t)
              *reinterpret_cast<uint32_t*>(dst + 8 * t + 2 * c) = pack_bf16x2(o[t][2 * h] * inv, o[t][2 * h + 1] * inv);
          } else {
            const RowFactors f = row_factors(l[h], m[h], u[h]);
            auto two = [&](float x, float y) {
              return pack_bf16x2(x * f.first * f.second, y * f.first * f.second);
            };
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int t = 0; t < NT; t += 8) {
                uint4 y;
                y.x = two(o[t][2 * h + j], o[t + 1][2 * h + j]);
                y.y = two(o[t + 2][2 * h + j], o[t + 3][2 * h + j]);
                y.z = two(o[t + 4][2 * h + j], o[t + 5][2 * h + j]);
                y.w = two(o[t + 6][2 * h + j], o[t + 7][2 * h + j]);
                *reinterpret_cast<uint4*>(dst + 2 * NT * c + j * NT + t) = y;
              }
          }
        } else {
          const long long idx = ((long long)blockIdx.x * 2 + slot) * R + lr;
          float* dst = a.part + idx * HD;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            dst[column(t)] = o[t][2 * h];
            dst[column(t) + kNext] = o[t][2 * h + 1];
          }
          if (c == 0) {
            if constexpr (B16)
              a.part_ml[idx] = make_float2(m[h], l[h]);
            else
              reinterpret_cast<float4*>(a.part_ml)[idx] = make_float4(m[h], u[h], l[h], 0.f);
          }
        }
      }
    }
    if (poisoned) {  // start the next query tile clean
      consumers_sync();
      for (int i = tid; i < HD; i += kThreads) bad[i] = Poison{0x7fffffff, 0x7fffffff, 0x7fffffff};
      consumers_sync();
    }
  };

  int stage = 0;
  uint32_t phase = 0;
  for (bool more = true; more; more = plan_next_item(a.plan, p, range, at)) {
    const int count = plan_here(range, at);
    start_item();
    paged_from = 0x7fffffff;
    for (int j = 0; j < count; ++j) {
      // a warp whose wait gives up keeps to the loop, and with it to the barriers
      // that the four warps share: later waits give up at once
      const bool got = __all_sync(
          0xffffffffu, mbar_wait_bounded(&sh.full[stage], phase, err, DEV_TIMEOUT_FULL, a.wp.limit_ns));
      const int k0 = (at.tile + j) * kKeys;
      if (got && k0 < seen_max) {  // some row sees the tile
        const uint32_t have = sh.with_page[stage];
        const bool all = k0 + kKeys <= seen_min && have == 15u;
        if (have != 0) paged_from = min(paged_from, k0 + 16 * (__ffs((int)have) - 1));
        const std::false_type no;
        const std::true_type yes;
        if constexpr (B16) {
          all ? add_tile(stage, k0, no, no) : add_tile(stage, k0, yes, no);
        } else if (wide || !(all ? add_tile(stage, k0, no, no) : add_tile(stage, k0, yes, no))) {
          add_tile(stage, k0, yes, yes);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stage]);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    // (a part of a cut item without tiles says that it has no sum)
    finish_item(at.tile == 0 && count == at.tiles, at.tile == 0 ? 1 : 0);
  }
}

// Up to 8 NB rows, NB 1 or 2, with the products turned round: S^T = K Q^T and O^T = V^T W^T,
// keys and value columns on the 16-row side, rows in 8-column tiles.  Each warp
// takes 16 of a tile's 64 keys for all rows.  The queries' fragments lie in
// shared memory in the order the lanes read them (with 16 rows they would be 32
// registers); weights turn from accumulators into B fragments by movmatrix.
template <int HD, int TYPE, int NB>
__global__ void __launch_bounds__(kThreads + 32, RowsCfg<HD, TYPE, NB>::BLOCKS)
    turned_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PagedArgs a,
                  const PagedView p) {
  using C = RowsCfg<HD, TYPE, NB>;
  constexpr bool B16 = C::B16;
  constexpr int R = 8 * NB;       // rows of a query tile
  constexpr int KS = HD / 16;     // steps of the first product, tiles of the second
  constexpr int NC = HD / 8;      // value columns of a lane's codes
  using Op = typename std::conditional<B16, bf16, f16>::type;
  constexpr float kNominal = B16 ? 0.f : 7.f, kRaise = kNominal + 8.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  __shared__ Poison bad[HD];
  __shared__ RowsShared<C> sh;
  // (read where they are needed: registers are short)
  __shared__ float scale_of_row[R];
  __shared__ int visible_to_row[R];
  __shared__ float sum_ref[B16 ? 1 : 4][R];  // as in rows_kernel
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = lane >> 2, c = lane & 3;
  const uint32_t sbase = smem_u32(smem);
  float* join = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
  uint2* queries = reinterpret_cast<uint2*>(smem + C::STAGES * C::STAGE + C::JOIN);  // [NB][KS][lane]
  int* err = &g_paged_err;

  for (int i = tid; i < HD; i += kThreads + 32) bad[i] = Poison{0x7fffffff, 0x7fffffff, 0x7fffffff};
  init_barriers<C>(sh);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  plan_and_keep(a, p, sh.scratch, sh.range);  // the block has met: barriers and notes are set up
  const PlanRange& range = sh.range;
  if (range.empty) return;
  if (warp == 4) {
    produce<C>(tm_k, tm_v, a, p, range, sh, smem);
    return;
  }

  PlanCursor at = range.first;
  // o[nb][t][i]: rows 8 nb + 2c + (i & 1), a value column for t and i >> 1
  float o[NB][KS][4];
  float m[NB][2], l[NB][2];
  int seen_min = 0, seen_max = 0;
  bool noted = false, wide = false;
  int paged_from = 0;

  auto start_item = [&]() {
    const int rows = at.n * a.plan.group;
    noted = wide = false;
    seen_min = plan_visible(at, at.qt * R / a.plan.group);
    seen_max = plan_visible(at, min(rows - 1, at.qt * R + R - 1) / a.plan.group);
    if (warp < NB) {  // this warp lays out the queries of 8 rows, a lane those of row r
      const int row = at.qt * R + 8 * warp + r, tok = row / a.plan.group;
      const bool valid = row < rows;
      if (c == 0) visible_to_row[8 * warp + r] = valid ? plan_visible(at, tok) : 0;
      const bf16* q = a.q + (long long)(at.row0 + tok) * a.q_stride + (at.head * a.plan.group + row % a.plan.group) * HD;
      uint2 w[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        if constexpr (B16) {  // elements 16 s + 2c, + 1 and 8 further
          const uint32_t* src = reinterpret_cast<const uint32_t*>(q) + 8 * s + c;
          w[s] = valid ? make_uint2(__ldg(src), __ldg(src + 4)) : make_uint2(0u, 0u);
        } else {  // step s of block s / 4: elements 64 (s / 4) + 16 c + 4 (s % 4) + 0..3, as the codes are read
          w[s] = valid ? __ldg(reinterpret_cast<const uint2*>(q) + 16 * (s >> 2) + 4 * c + (s & 3)) : make_uint2(0u, 0u);
        }
      }
      if constexpr (!B16) {
        float top = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint32_t x[2] = {w[s].x, w[s].y};
#pragma unroll
          for (int i = 0; i < 2; ++i)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xffff0000u))));
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // q * 2^up has its largest element in [2^14, 2^15)
        const int up = min(100, 14 - ((int)(__float_as_uint(top) >> 23) - 127));
        const float f = __uint_as_float((uint32_t)(127 + max(up, -126)) << 23);
        if (c == 0) scale_of_row[8 * warp + r] = a.scale_log2 / f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
          w[s] = make_uint2(pack_f16x2(__uint_as_float(w[s].x << 16) * f, __uint_as_float(w[s].x & 0xffff0000u) * f),
                            pack_f16x2(__uint_as_float(w[s].y << 16) * f, __uint_as_float(w[s].y & 0xffff0000u) * f));
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) queries[(warp * KS + s) * 32 + lane] = w[s];
    }
    consumers_sync();  // (the previous item's queries have been read, see its end)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[nb][j] = -INFINITY;
        l[nb][j] = 0.f;
      }
#pragma unroll
      for (int t = 0; t < KS; ++t) o[nb][t][0] = o[nb][t][1] = o[nb][t][2] = o[nb][t][3] = 0.f;
    }
  };

  // Value column of o[nb][t][i].
  auto column = [&](int t, int i) { return B16 ? 16 * t + r + 8 * (i >> 1) : NC * r + 2 * t + (i >> 1); };

  // The tile in `stage`: this warp's 16 keys.  A thread's scores are of keys
  // key0 and key0 + 8.  `mask`, `wide_form` and what is returned as in rows_kernel.
  auto add_tile = [&](int stage, int k0, auto mask, auto wide_form) {
    const uint32_t sk = sbase + stage * C::STAGE, sv = sk + C::POOL;
    const int kw = warp * 16;
    const bool paged = !mask() || (sh.with_page[stage] >> warp & 1u);
    auto piece_at = [&](int row, int piece) {
      if constexpr (C::LINE == 64) return row * 64 + ((piece ^ (row >> 1 & 3)) << 4);
      return (piece >> 3) * (kKeys * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
    };
    // the key of 8 read for matrix row r: with 2c and 2c ^ 5 for 2c and 2c + 1
    // no bank is met twice (codes; bf16 fragments are fixed by ldmatrix)
    auto key_of = [&](int row) { return B16 ? row : (row & 1 ? (row & 6) ^ 5 : row); };
    const int key0 = kw + key_of(r);
    float s[NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
    auto score_step = [&](int step, const uint32_t* k) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const uint2 q = queries[(nb * KS + step) * 32 + lane];
        mma16816<TYPE>(s[nb], k, q.x, q.y);
      }
    };
    if constexpr (B16) {
      const int row = kw + (lane & 7) + 8 * (lane >> 3 & 1);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t k[4];
        ldsm4(k, sk + piece_at(row, 2 * ks + (lane >> 4)));
        score_step(ks, k);
      }
    } else {
#pragma unroll
      for (int blk = 0; blk < HD / 64; ++blk) {
        const uint4 lo = lds128(sk + piece_at(key0, 4 * blk + c)), hi = lds128(sk + piece_at(key0 + 8, 4 * blk + c));
        const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, y[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t k[4] = {e4m3x2_to_f16x2(x[i]), e4m3x2_to_f16x2(y[i]), e4m3x2_to_f16x2(x[i] >> 16),
                                 e4m3x2_to_f16x2(y[i] >> 16)};
          score_step(4 * blk + i, k);
        }
      }
    }
    [[maybe_unused]] float kf[2] = {1.f, 1.f}, vf[2] = {1.f, 1.f}, ev[2] = {0.f, 0.f};
    [[maybe_unused]] bool beyond = false;
    if constexpr (!B16) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at_key = sk + 2 * C::POOL + key0 + 8 * h;
        const bool held = !mask() || (paged && k0 + key0 + 8 * h < seen_max);  // (else its bytes may be anything)
        const uint32_t kbyte = held ? lds_u8(at_key) : 127u, vbyte = held ? lds_u8(at_key + kKeys) : 127u;
        kf[h] = scale_of(kbyte);
        vf[h] = wide_form() ? scale_exponent(vbyte) : scale_of(vbyte);
        ev[h] = (float)((int)vbyte - 127);
        beyond |= !wide_form() && wide_scale(vbyte);
      }
    }
    // scores in log2 units, and whether a row's reference has to move: only
    // when a weight would pass 2^8 times its nominal largest (1, or 2^7 over
    // codes, whose fp16 weights end at 2^16), which spares most tiles the
    // shuffles and the rescaling
    bool moves = wide_form() || beyond;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = i >> 1, j = i & 1;  // key, row
        float x = s[nb][i] * (B16 ? a.scale_log2 : scale_of_row[8 * nb + 2 * c + j]);
        if constexpr (!B16) x *= kf[h];
        if (mask() && (k0 + key0 + 8 * h >= visible_to_row[8 * nb + 2 * c + j] || !paged)) x = -INFINITY;
        s[nb][i] = x;
        if constexpr (!B16) x += ev[h];
        moves |= x > m[nb][j] + kRaise;
      }
    }
    [[maybe_unused]] float uref[NB][2];
    if (__any_sync(0xffffffffu, moves)) {
      if (!B16 && !wide_form() && __any_sync(0xffffffffu, beyond)) return false;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        float corr[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float mx = B16 ? fmaxf(s[nb][j], s[nb][2 + j]) : fmaxf(s[nb][j] + ev[0], s[nb][2 + j] + ev[1]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
          const float next = fmaxf(m[nb][j], mx - kNominal), ref = next == -INFINITY ? 0.f : next;
          corr[j] = m[nb][j] == next ? 1.f : fast_exp2(m[nb][j] - ref);
          if constexpr (wide_form()) {
            const float from = wide ? sum_ref[warp][8 * nb + 2 * c + j] : m[nb][j];
            float up = fmaxf(from, fmaxf(s[nb][j], s[nb][2 + j]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, d));
            l[nb][j] *= from == up ? 1.f : fast_exp2(from - up);
            uref[nb][j] = up == -INFINITY ? 0.f : up;
            __syncwarp();
            if (r == 0) sum_ref[warp][8 * nb + 2 * c + j] = up;
          } else {
            l[nb][j] *= corr[j];
          }
          m[nb][j] = next;
        }
#pragma unroll
        for (int t = 0; t < KS; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nb][t][i] *= corr[i & 1];
      }
      if constexpr (wide_form()) {
        wide = true;
        __syncwarp();
      }
    }
    uint32_t w[NB][2];  // weights of 8 keys by 8 rows each, transposed into B fragments
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float e[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float x = s[nb][2 * h + j], above = x - (m[nb][j] == -INFINITY ? 0.f : m[nb][j]);
          if constexpr (wide_form()) {
            l[nb][j] += fast_exp2(x - uref[nb][j]);
            e[j] = fast_exp2(above + vf[h]);
            if (x == -INFINITY) e[j] = 0.f;  // a masked slot's scale byte may say infinity
          } else {
            e[j] = fast_exp2(above);
            l[nb][j] += e[j];
            if constexpr (!B16) e[j] *= vf[h];
          }
        }
        const uint32_t rows_of_key = pack2<Op>(e[0], e[1]);
        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(w[nb][h]) : "r"(rows_of_key));
      }
    }
    [[maybe_unused]] uint32_t x[4][B16 ? 1 : NC / 4];
    if constexpr (!B16) {
      // lane (r, c) takes columns NC r .. NC r + NC - 1 of the keys of matrix rows 2c, 2c + 1 of both 8s
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = kw + key_of(2 * c + (i & 1)) + 8 * (i >> 1);
        if constexpr (HD == 128) {
          const uint4 v = lds128(sv + piece_at(row, r));
          x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
        } else {
          const uint2 v = lds64(sv + piece_at(row, r >> 1) + 8 * (r & 1));
          x[i][0] = v.x, x[i][1] = v.y;
        }
      }
    }
#pragma unroll
    for (int t = 0; t < KS; ++t) {
      uint32_t v[4];  // columns column(t, 0), column(t, 2) of the keys of the first 8, then of the second
      if constexpr (B16) {
        const int row = kw + (lane & 7) + 8 * (lane >> 4);
        ldsm4t(v, sv + piece_at(row, 2 * t + (lane >> 3 & 1)));
      } else {
        const uint32_t sel = t & 1 ? 0x7362u : 0x5140u;
        const uint32_t lo = __byte_perm(x[0][t / 2], x[1][t / 2], sel), hi = __byte_perm(x[2][t / 2], x[3][t / 2], sel);
        v[0] = e4m3x2_to_f16x2(lo), v[1] = e4m3x2_to_f16x2(lo >> 16);
        v[2] = e4m3x2_to_f16x2(hi), v[3] = e4m3x2_to_f16x2(hi >> 16);
      }
      if (mask()) {  // as `clean` in rows_kernel
        constexpr uint32_t E = B16 ? 0x7f80u : 0x7c00u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int col = column(t, 2 * (i & 1));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int key = k0 + kw + key_of(2 * c + half) + 8 * (i >> 1);
            const uint32_t y = v[i] >> (16 * half) & 0xffffu;
            const bool unseen = key >= seen_max || !paged;
            if (!unseen && ((y & E) != E || k0 + kKeys <= seen_min)) continue;
            if (!unseen) {
              int* slot = (y & ~(E | 0x8000u)) != 0 ? &bad[col].nan : (y & 0x8000u) ? &bad[col].neg : &bad[col].pos;
              atomicMin(slot, key);
              noted = true;
            }
            v[i] &= half ? 0x0000ffffu : 0xffff0000u;
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma16816<TYPE>(o[nb][t], v, w[nb][0], w[nb][1]);
    }
    return true;
  };

  // Joins the four warps' sums and writes the query tile's rows, or its
  // partial sums.  Each warp brings its sums to the common reference; then four
  // tiles of value columns at a time pass through shared memory, each warp
  // adding up one of the four and writing it.
  auto finish_item = [&](bool whole, int slot) {
    float2* stats = reinterpret_cast<float2*>(join);  // [warp][row] reference, sum
    [[maybe_unused]] float* refs = join + 8 * R;      // [warp][row] codes: the sum's reference
    [[maybe_unused]] float u[NB][2];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nb][j] += __shfl_xor_sync(0xffffffffu, l[nb][j], d);
        m[nb][j] = seen_reference(m[nb][j], paged_from < visible_to_row[8 * nb + 2 * c + j]);
        if (r == 0) {
          const int row = 8 * nb + 2 * c + j;
          stats[warp * R + row] = make_float2(m[nb][j], l[nb][j]);
          if constexpr (!B16) refs[warp * R + row] = wide ? sum_ref[warp][row] : m[nb][j];
        }
      }
    const bool poisoned = consumers_any(noted);  // every warp has noted its non-finite values, and read the queries
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float own[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float2 st[4];
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          st[k] = stats[k * R + 8 * nb + 2 * c + j];
          top = fmaxf(top, st[k].x);
        }
        const float ref = top == -INFINITY ? 0.f : top;
        l[nb][j] = 0.f;
        if constexpr (B16) {
#pragma unroll
          for (int k = 0; k < 4; ++k) l[nb][j] += st[k].y * fast_exp2(st[k].x - ref);
        } else {
          float of[4];
          u[nb][j] = -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            of[k] = refs[k * R + 8 * nb + 2 * c + j];
            u[nb][j] = fmaxf(u[nb][j], of[k]);
          }
          const float uref = u[nb][j] == -INFINITY ? 0.f : u[nb][j];
#pragma unroll
          for (int k = 0; k < 4; ++k) l[nb][j] += st[k].y * fast_exp2(of[k] - uref);
        }
        own[j] = fast_exp2(m[nb][j] - ref);
        m[nb][j] = top;
      }
#pragma unroll
      for (int t = 0; t < KS; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nb][t][i] *= own[i & 1];
    }
    const int rows = at.n * a.plan.group;
    auto out_of = [&](int row) {
      const int tok = row / a.plan.group;
      return a.out + (long long)(at.row0 + tok) * a.out_stride + (at.head * a.plan.group + row % a.plan.group) * HD;
    };
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      RowFactors f[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        f[j] = row_factors(l[nb][j], m[nb][j], B16 ? m[nb][j] : u[nb][j]);
#pragma unroll
      for (int t0 = 0; t0 < KS; t0 += 4) {
        consumers_sync();  // the statistics, or the tiles before, have been read
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) join[(warp * 16 + 4 * t + i) * 32 + lane] = o[nb][t0 + t][i];
        consumers_sync();
        const int t = t0 + warp;
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          y[i] = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) y[i] += join[(k * 16 + 4 * warp + i) * 32 + lane];
          if (poisoned) y[i] += poison_of(bad[column(t, i)], visible_to_row[8 * nb + 2 * c + (i & 1)]);
          if (whole) y[i] *= f[i & 1].first;
          if (whole && !B16) y[i] *= f[i & 1].second;
        }
        if (whole && B16) {
          // columns r (and r + 8) of rows 2c, 2c + 1 -> row r, columns 2c, 2c + 1
          const int row = at.qt * R + 8 * nb + r;
          bf16* dst = out_of(min(row, rows - 1)) + 16 * t + 2 * c;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t z = pack_bf16x2(y[2 * h], y[2 * h + 1]);
            asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(z) : "r"(z));
            if (row < rows) *reinterpret_cast<uint32_t*>(dst + 8 * h) = z;
          }
          continue;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int lr = 8 * nb + 2 * c + j, row = at.qt * R + lr;
          if (row >= rows) continue;
          if (whole) {
            *reinterpret_cast<uint32_t*>(out_of(row) + column(t, 0)) = pack_bf16x2(y[j], y[2 + j]);
          } else {
            float* dst = a.part + (((long long)blockIdx.x * 2 + slot) * R + lr) * HD;
            dst[column(t, 0)] = y[j];
            dst[column(t, 2)] = y[2 + j];
          }
        }
      }
      if (!whole && warp == 0 && r == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int lr = 8 * nb + 2 * c + j;
          if (at.qt * R + lr >= rows) continue;
          const long long idx = ((long long)blockIdx.x * 2 + slot) * R + lr;
          if constexpr (B16)
            a.part_ml[idx] = make_float2(m[nb][j], l[nb][j]);
          else
            reinterpret_cast<float4*>(a.part_ml)[idx] = make_float4(m[nb][j], u[nb][j], l[nb][j], 0.f);
        }
      }
    }
    if (poisoned) {  // start the next query tile clean
      consumers_sync();
      for (int i = tid; i < HD; i += kThreads) bad[i] = Poison{0x7fffffff, 0x7fffffff, 0x7fffffff};
      consumers_sync();
    }
  };

  int stage = 0;
  uint32_t phase = 0;
  for (bool more = true; more; more = plan_next_item(a.plan, p, range, at)) {
    const int count = plan_here(range, at);
    start_item();
    paged_from = 0x7fffffff;
    for (int j = 0; j < count; ++j) {
      const bool got = __all_sync(
          0xffffffffu, mbar_wait_bounded(&sh.full[stage], phase, err, DEV_TIMEOUT_FULL, a.wp.limit_ns));
      const int k0 = (at.tile + j) * kKeys;
      if (got && k0 < seen_max) {  // some row sees the tile
        const uint32_t have = sh.with_page[stage];
        const bool all = k0 + kKeys <= seen_min && have == 15u;
        if (have != 0) paged_from = min(paged_from, k0 + 16 * (__ffs((int)have) - 1));
        const std::false_type no;
        const std::true_type yes;
        if constexpr (B16) {
          all ? add_tile(stage, k0, no, no) : add_tile(stage, k0, yes, no);
        } else if (wide || !(all ? add_tile(stage, k0, no, no) : add_tile(stage, k0, yes, no))) {
          add_tile(stage, k0, yes, yes);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.empty[stage]);
      if (++stage == C::STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    finish_item(at.tile == 0 && count == at.tiles, at.tile == 0 ? 1 : 0);
  }
}

// Adds the partial sums of the query tile that block boundary blockIdx.x + 1
// falls into, if it is the first boundary inside that tile; kJoinRows rows of
// it a block.  The parts of a row are dealt to 8 or 16 groups of threads, each
// thread taking 4 columns of 4 rows at a time, so that an item cut into many
// parts is a few loads deep; the groups' sums meet in shared memory in group
// order, so the order of all additions is fixed.  TWO: the parts of an e4m3
// cache's few-row kernels, whose sums of weights have a reference of their own.
constexpr int kJoinRows = 16;
template <int HD, bool TWO>
__global__ void __launch_bounds__(256, TWO ? 3 : 4) join_kernel(const PagedArgs a, const PagedView p) {
  constexpr int COLS = HD / 4, GROUPS = 256 / COLS, DEEP = 4;
  __shared__ float4 sums[GROUPS][DEEP][COLS];
  __shared__ float2 stats[GROUPS][DEEP];  // reference, sum of weights
  __shared__ float refs[TWO ? GROUPS : 1][DEEP];  // the sum's reference
  // every block waits, also those with nothing to do: this kernel's end then
  // says that both have ended
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the last block seldom has rows to join: its look at the error word delays nobody
  if (blockIdx.x + 1 == gridDim.x && blockIdx.y == 0 && threadIdx.x == 0 && *a.own_err != 0)
    atomicCAS(a.err, 0, atomicExch(a.own_err, 0));
  const int i = (int)blockIdx.x + 1;
  if (i >= a.plan.blocks) return;
  const PlanRange range = a.plans[i];
  const PlanCursor prev = a.plans[i - 1].first;
  if (range.empty) return;
  const PlanCursor at = range.first;
  if (at.tile == 0) return;  // the boundary is between two items
  if (plan_same_item(prev, at) && prev.tile > 0) return;  // an earlier boundary lies inside too
  const int R = a.plan.rows, rows = min(R, at.n * a.plan.group - at.qt * R);
  const int row0 = (int)blockIdx.y * kJoinRows, row1 = min(rows, row0 + kJoinRows);
  const int last = plan_block_of(range, range.item_end - 1);
  const int col = threadIdx.x % COLS, grp = threadIdx.x / COLS;
  for (int base = row0; base < row1; base += DEEP) {
    float top[DEEP], l[DEEP];
    [[maybe_unused]] float u[DEEP];
    float4 s[DEEP];
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      top[d] = u[d] = -INFINITY;
      l[d] = 0.f;
      s[d] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k = i - 1 + grp; k <= last; k += GROUPS) {
      float2 ml[DEEP];
      [[maybe_unused]] float part_u[DEEP];
      float4 v[DEEP];
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        const long long idx = ((long long)k * 2 + (k == i - 1 ? 1 : 0)) * R + min(base + d, row1 - 1);
        if constexpr (TWO) {
          const float4 st = reinterpret_cast<const float4*>(a.part_ml)[idx];
          ml[d] = make_float2(st.x, st.z);
          part_u[d] = st.y;
        } else {
          ml[d] = a.part_ml[idx];
        }
        v[d] = *reinterpret_cast<const float4*>(a.part + idx * HD + 4 * col);
      }
#pragma unroll
      for (int d = 0; d < DEEP; ++d) {
        const float m = fmaxf(top[d], ml[d].x), ref = m == -INFINITY ? 0.f : m;
        const float f0 = fast_exp2(top[d] - ref), f1 = fast_exp2(ml[d].x - ref);
        top[d] = m;
        if constexpr (TWO) {
          const float up = fmaxf(u[d], part_u[d]), uref = up == -INFINITY ? 0.f : up;
          l[d] = l[d] * fast_exp2(u[d] - uref) + ml[d].y * fast_exp2(part_u[d] - uref);
          u[d] = up;
        } else {
          l[d] = l[d] * f0 + ml[d].y * f1;
        }
        s[d].x = s[d].x * f0 + v[d].x * f1;
        s[d].y = s[d].y * f0 + v[d].y * f1;
        s[d].z = s[d].z * f0 + v[d].z * f1;
        s[d].w = s[d].w * f0 + v[d].w * f1;
      }
    }
    __syncthreads();  // the previous rows have been read
#pragma unroll
    for (int d = 0; d < DEEP; ++d) {
      sums[grp][d][col] = s[d];
      if (col == 0) stats[grp][d] = make_float2(top[d], l[d]);
      if (TWO && col == 0) refs[grp][d] = u[d];
    }
    __syncthreads();
    if (grp < DEEP && base + grp < row1) {
      float m = -INFINITY;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) m = fmaxf(m, stats[g][grp].x);
      const float ref = m == -INFINITY ? 0.f : m;
      [[maybe_unused]] float up = -INFINITY, uref = 0.f;
      if constexpr (TWO) {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) up = fmaxf(up, refs[g][grp]);
        uref = up == -INFINITY ? 0.f : up;
      }
      float o[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const float2 st = stats[g][grp];
        const float4 v = sums[g][grp][col];
        const float f = fast_exp2(st.x - ref);
        sum += st.y * (TWO ? fast_exp2(refs[TWO ? g : 0][grp] - uref) : f);
        o[0] += f * v.x, o[1] += f * v.y, o[2] += f * v.z, o[3] += f * v.w;
      }
      const int row = at.qt * R + base + grp;
      const int tok = row / a.plan.group, head = at.head * a.plan.group + row % a.plan.group;
      const RowFactors f = row_factors(sum, m, TWO ? up : m);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] *= f.first;
      if constexpr (TWO) {
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] *= f.second;
      }
      bf16* dst = a.out + (long long)(at.row0 + tok) * a.out_stride + head * HD + 4 * col;
      *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
    }
  }
}

template <typename C, typename Kernel>
armt_status launch_few(Kernel kernel, DeviceOnce& once, const PagedArgs& a, const PagedView& p,
                       const armt_kv_cache& cache, cudaStream_t st) {
  if (once.need(a.device)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return launch_status(e, "paged attention set-up");
    once.set(a.device);
  }
  CUtensorMap tm_k, tm_v;
  if (!encode_pool(&tm_k, p.k, cache, kKeys) || !encode_pool(&tm_v, p.v, cache, kKeys))
    return refuse(ARMT_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  kernel<<<a.plan.blocks, kThreads + 32, C::SMEM, st>>>(tm_k, tm_v, a, p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_join(a, p, cache.head_dim, !C::B16, st);
  return launch_status(e, "paged attention");
}
template <int HD, int TYPE, int WM>
armt_status launch_rows(const PagedArgs& a, const PagedView& p, const armt_kv_cache& cache, cudaStream_t st) {
  static DeviceOnce once;
  return launch_few<RowsCfg<HD, TYPE, 0, WM>>(rows_kernel<HD, TYPE, WM>, once, a, p, cache, st);
}
template <int HD, int TYPE, int NB>
armt_status launch_turned(const PagedArgs& a, const PagedView& p, const armt_kv_cache& cache, cudaStream_t st) {
  static DeviceOnce once;
  return launch_few<RowsCfg<HD, TYPE, NB>>(turned_kernel<HD, TYPE, NB>, once, a, p, cache, st);
}
template <int HD, int TYPE>
armt_status launch_shape(int rows, const PagedArgs& a, const PagedView& p, const armt_kv_cache& cache, cudaStream_t st) {
  switch (rows) {
    case 8: return launch_turned<HD, TYPE, 1>(a, p, cache, st);
    case 16: return launch_turned<HD, TYPE, 2>(a, p, cache, st);
    case 32: return launch_rows<HD, TYPE, 2>(a, p, cache, st);
  }
  if constexpr (HD == 64) return launch_rows<HD, TYPE, 4>(a, p, cache, st);
  return refuse(ARMT_ERR_UNSUPPORTED, "no kernel for this shape");
}
template <int HD, int TYPE>
int few_blocks(int rows) {
  if (rows <= 16) return rows == 8 ? RowsCfg<HD, TYPE, 1>::BLOCKS : RowsCfg<HD, TYPE, 2>::BLOCKS;
  return rows == 32 ? RowsCfg<HD, TYPE, 0, 2>::BLOCKS : RowsCfg<HD, TYPE, 0, 4>::BLOCKS;
}

// How a call is cut up: rows of a query tile, and blocks.  Both depend on
// sizes the host knows; what the arrays hold only moves the block boundaries.
struct Shape {
  bool tiles;  // the tensor-core kernel for many rows
  int rows;    // of a query tile
  int blocks;  // of the grid
  int64_t bytes;
};

template <int HD>
int few_blocks(bool b16, int rows) {
  return b16 ? few_blocks<HD, ARMT_CACHE_BF16>(rows) : few_blocks<HD, ARMT_CACHE_E4M3>(rows);
}

// Workspace for query tiles of up to `rows` rows of a kv head: the most that any
// such call over either cache type needs, so that one sized for the largest batch
// serves all others of the same heads.
int64_t workspace_bytes(int hd, int group, int64_t rows, int sms) {
  auto need = [&](int blocks, int tile) {
    return (int64_t)blocks * (2 * tile * (hd + 4) * 4 + (int64_t)sizeof(PlanRange));
  };
  int64_t most = 0;
  for (int tile = 8; tile <= (hd == 128 ? 32 : 64); tile *= 2) {
    for (bool b16 : {false, true})
      most = std::max(most, need((hd == 64 ? few_blocks<64>(b16, tile) : few_blocks<128>(b16, tile)) * sms, tile));
    if (rows <= tile) return most;
  }
  return std::max(most, need(sms, tile_rows(group)));
}

Shape shape_of(const armt_kv_cache& c, const armt_paged_batch& b, int group, int sms) {
  Shape s;
  const int64_t rows = (b.max_new < b.n_rows ? (int64_t)b.max_new : b.n_rows) * group;
  const bool b16 = c.type == ARMT_CACHE_BF16;
  // Past 32 rows of head_dim 128 the tensor-core kernel is the faster one over
  // either type.  bf16, 16 sequences of 10 or 14 tokens, 32 / 8 heads, contexts to
  // 8K: 98 us for 113; 2 sequences 38 for 50.  e4m3, 9 / 12 / 16 tokens: 16
  // sequences 131 / 133 / 132 for 147 / 155 / 162, 2 sequences 55 / 56 / 56 for 79 /
  // 84 / 87, 64 sequences 425 / 425 / 427 for 457 / 471 / 496 (the few-row kernel's
  // sums spill there); only many long contexts go the other way (16 of 30,000
  // tokens: 638 for 550).  The weights are then bf16 for fp16.  With head_dim 64,
  // where its softmax is twice the work of its products, past 64 rows (83 for 60;
  // 30 for 39).
  s.tiles = rows > (c.head_dim == 128 ? 32 : 64);
  s.rows = s.tiles ? tile_rows(group) : rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
  s.blocks = sms;
  if (!s.tiles) s.blocks *= c.head_dim == 64 ? few_blocks<64>(b16, s.rows) : few_blocks<128>(b16, s.rows);
  s.bytes = workspace_bytes(c.head_dim, group, rows, sms);
  return s;
}

armt_status check_attention(const armt_kv_cache* cache, const armt_paged_batch* batch, int32_t n_q_heads) {
  armt_status s;
  if ((s = check_cache(cache)) != ARMT_OK || (s = check_batch(batch, cache)) != ARMT_OK) return s;
  if (n_q_heads <= 0) return refuse(ARMT_ERR_ARG, "sizes must be positive");
  if (n_q_heads % cache->n_kv_heads != 0)
    return refuse(ARMT_ERR_SHAPE, "n_q_heads must be a multiple of n_kv_heads");
  if (n_q_heads / cache->n_kv_heads > 64)
    return refuse(ARMT_ERR_UNSUPPORTED, "at most 64 query heads for a kv head");
  if (batch->n_rows * n_q_heads > 0x7fffffffll)
    return refuse(ARMT_ERR_SHAPE, "n_rows * n_q_heads must be at most 2^31 - 1");
  return ARMT_OK;
}

}  // namespace

cudaError_t launch_join(const PagedArgs& a, const PagedView& p, int head_dim, bool two, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max(1, a.plan.blocks - 1), (unsigned)((a.plan.rows + kJoinRows - 1) / kJoinRows));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (two) return cudaLaunchKernelEx(&cfg, head_dim == 64 ? join_kernel<64, true> : join_kernel<128, true>, a, p);
  return cudaLaunchKernelEx(&cfg, head_dim == 64 ? join_kernel<64, false> : join_kernel<128, false>, a, p);
}

}  // namespace armt

using namespace armt;

extern "C" ARMT_API armt_status armt_paged_attention_workspace(const armt_kv_cache* cache,
                                                               const armt_paged_batch* batch, int32_t n_q_heads,
                                                               int64_t* bytes) {
  return guarded([&]() -> armt_status {
    if (bytes == nullptr) return refuse(ARMT_ERR_ARG, "NULL argument");
    armt_status s = check_attention(cache, batch, n_q_heads);
    if (s != ARMT_OK) return s;
    int dev = 0, sms = 0;
    if ((s = ready_device(&dev, &sms)) != ARMT_OK) return s;
    *bytes = shape_of(*cache, *batch, n_q_heads / cache->n_kv_heads, sms).bytes;
    return ARMT_OK;
  });
}

extern "C" ARMT_API armt_status armt_paged_attention_bf16(const void* q, int64_t q_stride, const armt_kv_cache* cache,
                                                          const armt_paged_batch* batch, int32_t n_q_heads,
                                                          float scale, void* out, int64_t out_stride, void* workspace,
                                                          int64_t workspace_bytes, void* stream) {
  return guarded([&]() -> armt_status {
    armt_status s = check_attention(cache, batch, n_q_heads);
    if (s != ARMT_OK) return s;
    const int64_t width = (int64_t)n_q_heads * cache->head_dim;
    if ((s = check_rows(q, batch->n_rows, q_stride, width, "q")) != ARMT_OK || (s = check_rows(out, batch->n_rows, out_stride, width, "out")) != ARMT_OK)
      return s;
    if (workspace == nullptr) return refuse(ARMT_ERR_ARG, "NULL argument");
    if (misaligned16(workspace)) return refuse(ARMT_ERR_ARG, "pointers must be 16-byte aligned");
    if (!(scale > 0.f) || !(scale < 2.0e38f)) return refuse(ARMT_ERR_ARG, "scale must be positive and below 2e38");
    int dev = 0, sms = 0;
    if ((s = ready_device(&dev, &sms)) != ARMT_OK) return s;
    const int group = n_q_heads / cache->n_kv_heads;
    const Shape shape = shape_of(*cache, *batch, group, sms);
    if (workspace_bytes < shape.bytes)
      return refuse(ARMT_ERR_SHAPE, "workspace of " + std::to_string(workspace_bytes) + " bytes, " +
                                        std::to_string(shape.bytes) + " needed");
    if (batch->n_rows == 0) return ARMT_OK;
    PagedArgs a;
    a.q = static_cast<const bf16*>(q);
    a.out = static_cast<bf16*>(out);
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.plan.group = group;
    a.plan.rows = shape.rows;
    a.plan.blocks = shape.blocks;
    a.plan.keys = kKeys;
    a.plan.fixed = kFixedKeys;
    a.plan.least = 2;
    a.wp = wait_policy_from_env();
    a.device = dev;
    if ((s = block_error_word(dev, &a.err)) != ARMT_OK) return s;
    static DeviceSymbol word;
    const cudaError_t e = word.find(g_paged_err, dev, &a.own_err);
    if (e != cudaSuccess) return launch_status(e, "paged attention set-up");
    a.part = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(a.part + (int64_t)shape.blocks * 2 * a.plan.rows * cache->head_dim);
    a.plans = reinterpret_cast<PlanRange*>(a.part_ml + (int64_t)shape.blocks * 4 * a.plan.rows);
    const PagedView p = paged_view(*cache, *batch);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (shape.tiles) return launch_tiles(a, p, *cache, n_q_heads, st);
    if (cache->type == ARMT_CACHE_BF16)
      return cache->head_dim == 64 ? launch_shape<64, ARMT_CACHE_BF16>(shape.rows, a, p, *cache, st)
                                   : launch_shape<128, ARMT_CACHE_BF16>(shape.rows, a, p, *cache, st);
    return cache->head_dim == 64 ? launch_shape<64, ARMT_CACHE_E4M3>(shape.rows, a, p, *cache, st)
                                 : launch_shape<128, ARMT_CACHE_E4M3>(shape.rows, a, p, *cache, st);
  });
}
