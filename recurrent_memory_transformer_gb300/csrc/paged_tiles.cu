// Attention of many new rows over the paged cache, on tcgen05.
//
// A chunk of a prompt against its context: the products carry it
// (4 hd flops a row pair), so both run on the tensor cores out of shared
// memory and tensor memory.  A block owns an SM and works on an item of two
// query tiles ("slots") of up to 128 rows -- (token, head of the group) pairs,
// so grouped heads share each key tile -- against the item's key tiles of 128:
//
//   warp 8       producer: page table, TMA of Q (both slots) and of K_j, V_j
//                into a ring of buffers, in the order the products use them
//   warp 9       issues S_s = Q_s K_j^T (128 x 128, TMEM columns 128 s ...)
//                and O_s += P_s V_j (TMEM columns 256 + 128 s ...)
//   warps 0..3   softmax of slot 0, one thread a row; warps 4..7 of slot 1
//   warps 10..   clean V tiles that not every row sees; over an e4m3 cache
//                they also expand K and V to bf16, from buffers of their own
//                (code * 2^e is exact in bf16, so nothing is lost here)
//
// While one slot's scores go through the softmax the tensor core works for
// the other: PV_0(j), S_0(j+1), PV_1(j), S_1(j+1), ...  The weights P_s go
// back into tensor memory over the scores they came from (64 of the 128
// columns) and are the A operand there; V is used as it lies in the cache,
// keys by head_dim, as an MN-major B operand, so nothing is transposed.  The
// tensor core runs its products in the order they were issued: once S_s(j+1)
// has arrived, PV_s(j) has ended, and O_s may be touched until P_s(j+1) is
// handed over.  A row's reference maximum moves only when a tile's maximum
// passes it by more than 2^8, which makes rescaling O rare.
//
// What is held in fewer than 32 bits: the weights, rounded to bf16 (2^-8 of each,
// at any scale) because both operands of a product have one type and V is bf16;
// their sum is taken in fp32 before that, the references and O are fp32.  Against
// 64 bits the outputs are off by 0.0023 of their size, 0.0017 of it their own
// rounding to bf16.
//
// Blocks take equal shares of the list of tiles; see paged_plan.cuh.
#include <type_traits>

#include "paged_attn.cuh"
#include "paged_notes.h"
#include "register_split.h"

namespace armt {
namespace {

constexpr int kKeys = 128;
constexpr int kSoftmaxThreads = 256;

template <int HD, int TYPE>
struct TileCfg {
  static constexpr bool B16 = TYPE == ARMT_CACHE_BF16;
  // Cleaning alone is little work for two warps; expanding takes six (2 x
  // 1,024 rows over 16K, 680 us now: 631 for 685 with four when both were there),
  // and then the softmax warps need registers that the others give back.  (With four and the exchange
  // the bf16 kernel was a tenth slower, 533 us for 479.)
  static constexpr int CLEAN_WARP = 10, CLEAN_WARPS = B16 ? 2 : 6;
  static constexpr int THREADS = 32 * (CLEAN_WARP + CLEAN_WARPS);
  static constexpr int LAUNCH_REGS = B16 ? 168 : 128;
  static constexpr int SOFTMAX_REGS = 168, OTHER_REGS = 88;  // e4m3: 256 x 168 + 256 x 88 = 512 x 128
  static_assert(B16 || split_fits(LAUNCH_REGS, THREADS, kSoftmaxThreads, SOFTMAX_REGS, OTHER_REGS),
                "the register split must fit what the block is launched with");
  static constexpr int ATOMS = HD / 64;       // 128-byte wide parts of a bf16 row
  static constexpr int BUF = kKeys * HD * 2;  // a tile of Q, K or V as bf16
  static constexpr int RING = HD == 128 ? (B16 ? 5 : 3) : (B16 ? 8 : 4);
  static constexpr int CODES = kKeys * HD;    // a tile of codes
  static constexpr int RAW = B16 ? 1 : HD == 128 ? 3 : 6;  // buffers of codes (bf16: unused)
  static constexpr int RAW_BYTES = B16 ? 0 : RAW * (CODES + kKeys);  // with their scale bytes, after all codes
  static constexpr int BAD = HD * 12;
  static constexpr int SMEM = 1024 + (2 + RING) * BUF + RAW_BYTES + BAD + 512;
};

template <typename C>
__device__ __forceinline__ void give_registers() {
  if constexpr (!C::B16) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
}
template <typename C>
__device__ __forceinline__ void take_registers() {
  if constexpr (!C::B16) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
}

// Set by a bounded wait that gave up; the joining kernel passes it on.  (A word
// of the module's own: a pointer among the arguments costs the softmax warps
// registers that they spill, 2 x 1,024 rows over 16K 474 us -> 486, e4m3 head_dim
// 64 485 -> 507.)
__device__ int g_tiles_err;

// Barriers, after the ring in shared memory.
template <int RING, int RAW>
struct TileBars {
  uint64_t full[RING], empty[RING], ready[RING];  // bf16 buffers: landed (bf16 caches), free, fit for use
  uint64_t raw_full[RAW], raw_empty[RAW];         // buffers of codes
  uint64_t q_full, q_empty, s_full[2], p_ready[2], o_full[2], epilogue, drain;
  uint32_t tmem;
  int any_bad;
  PlanRange range;
  uint32_t with_page[16];  // of tile t at t % 16: 8 bits, which 16-key groups have a page
  int paged_from[4];       // of item i at i % 4: the first key, in this block's part, that has a page
};

// D[tmem] (+)= A[tmem] * B[smem], kind::f16.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Descriptor of a B operand whose N (64 bf16 = 128 bytes) lies contiguous, as
// TMA writes it with 128-byte swizzling: 8 keys are 1,024 bytes, the next 64
// columns of N `atom` bytes on.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t atom) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(atom >> 4) << 16;   // leading byte offset: along N
  d |= (uint64_t)(1024u >> 4) << 32;  // stride byte offset: along K
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

#define ARMT_TMEM_REGS32(r)                                                                                        \
  "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),       \
      "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),        \
      "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),       \
      "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])

// 32 columns of this warp's lanes, without waiting for them.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : ARMT_TMEM_REGS32(r)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int HD, int TYPE>
__global__ void __launch_bounds__(TileCfg<HD, TYPE>::THREADS, 1)
    tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const PagedArgs a, const PagedView p, const int slot_tokens) {
  using C = TileCfg<HD, TYPE>;
  constexpr bool B16 = C::B16;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = base;
  uint8_t* ring = base + 2 * C::BUF;
  uint8_t* raw = ring + C::RING * C::BUF;  // RAW buffers of codes, then RAW x 128 scale bytes
  Poison* bad = reinterpret_cast<Poison*>(raw + C::RAW_BYTES);
  using Bars = TileBars<C::RING, C::RAW>;
  Bars& bar = *reinterpret_cast<Bars*>(raw + C::RAW_BYTES + C::BAD);
  static_assert(sizeof(Bars) <= 512 && sizeof(PlanScratch) <= C::BUF, "shared memory layout");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int* err = &g_tiles_err;
  const uint64_t limit = a.wp.limit_ns;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  PlanRange& range = bar.range;
  plan_and_keep(a, p, *reinterpret_cast<PlanScratch*>(ring), range);
  if (range.empty) return;
  for (int i = tid; i < HD; i += C::THREADS) bad[i] = Poison{0x7fffffff, 0x7fffffff, 0x7fffffff};
  if (tid == 0) {
    for (int i = 0; i < C::RING; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
      mbar_init(&bar.ready[i], C::CLEAN_WARPS);
    }
    for (int i = 0; i < C::RAW; ++i) {
      mbar_init(&bar.raw_full[i], 1);
      mbar_init(&bar.raw_empty[i], C::CLEAN_WARPS);
    }
    mbar_init(&bar.q_full, 1);
    mbar_init(&bar.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.p_ready[s], 4);
      mbar_init(&bar.o_full[s], 1);
    }
    mbar_init(&bar.epilogue, 8);
    mbar_init(&bar.drain, 1);
    bar.any_bad = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  fence_proxy_async_smem();
  __syncthreads();  // the plan's scratch, where the ring will be, is done with
  if (warp == 9) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;

  PlanCursor at = range.first;
  if (warp == 8) {
    // ------------------------------------------------------- producer --
    give_registers<C>();
    constexpr int BUFS = B16 ? C::RING : C::RAW;
    uint64_t* const full = B16 ? bar.full : bar.raw_full;
    uint64_t* const empty = B16 ? bar.empty : bar.raw_empty;
    const int run = min(1 << p.page_shift, kKeys), runs = kKeys / run;
    const uint32_t run_bits = (1u << (run / 16)) - 1u;
    struct {
      int ids, at, b;
    } look[2] = {{-1, 0, -1}, {-1, 0, -1}};  // page ids of 32 runs, for K and for V (which trails)
    int n = 0, items = 0, tiles = 0, paged_from = 0;
    bool ok = true;
    // the copies of tile `tile` of K (pool 0) or V (1) into the next buffer
    auto load = [&](int pool, int tile, int count) {
      const int b = n % BUFS, k0 = tile * kKeys;
      ok = n != a.wp.stall_after &&
           (n < BUFS || mbar_wait_bounded(&empty[b], (uint32_t)((n / BUFS - 1) & 1), err, DEV_TIMEOUT_EMPTY, limit));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      auto& l = look[pool];
      if (at.b != l.b || k0 < l.at || k0 + kKeys - l.at > 32 * run) {
        const long long key = (long long)k0 + run * lane;
        l.ids = key < at.kv ? paged_page(p, at.b, key) : -1;
        l.at = k0;
        l.b = at.b;
      }
      const int page = __shfl_sync(0xffffffffu, l.ids, ((k0 - l.at) / run + lane) & 31);
      const bool mine = lane < runs && page >= 0;
      const uint32_t have = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) {
        if (pool == 0) {
          uint32_t groups = 0;
          for (int j = 0; j < runs; ++j) groups |= (have >> j & 1u) * (run_bits << (j * run / 16));
          bar.with_page[count % 16] = groups;
          if (groups != 0) paged_from = min(paged_from, k0 + 16 * (__ffs((int)groups) - 1));
          bar.paged_from[(items - 1) % 4] = paged_from;
        }
        mbar_arrive_expect_tx(&full[b], (uint32_t)(__popc(have) * run * (B16 ? HD * 2 : HD + 1)));
      }
      __syncwarp();
      if (mine) {
        const int key = lane * run, slot = (k0 + key) & ((1 << p.page_shift) - 1);
        const CUtensorMap* tm = pool == 0 ? &tm_k : &tm_v;
        if constexpr (B16) {
#pragma unroll
          for (int t = 0; t < C::ATOMS; ++t)
            tma_load_3d(ring + b * C::BUF + t * (kKeys * 128) + key * 128, tm, t * 64, slot, page * p.hkv + at.head,
                        &full[b]);
        } else {
          tma_load_3d(raw + b * C::CODES + key * HD, tm, 0, slot, page * p.hkv + at.head, &full[b]);
          bulk_load(raw + C::RAW * C::CODES + b * kKeys + key,
                    (pool == 0 ? p.k_scale : p.v_scale) + paged_row(p, page, at.head, slot), run, &full[b]);
        }
      }
      ++n;
    };
    for (bool more = true; ok && more; more = plan_next_item(a.plan, p, range, at)) {
      const int count = plan_here(range, at);
      if (count == 0) continue;  // an empty part of a cut item: the softmax warps say so
      if (lane == 0) {
        ok = items == 0 || mbar_wait_bounded(&bar.q_empty, (uint32_t)((items - 1) & 1), err, DEV_TIMEOUT_EMPTY, limit);
        if (ok) {
          // rows of a box: slot_tokens tokens of `group` heads; past the batch's rows it is filled with zeros
          mbar_arrive_expect_tx(&bar.q_full, (uint32_t)(2 * slot_tokens * a.plan.group * HD * 2));
          for (int s = 0; s < 2; ++s)
            for (int t = 0; t < C::ATOMS; ++t)
              tma_load_3d(sQ + s * C::BUF + t * (128 * 128), &tm_q, t * 64, at.head * a.plan.group,
                          at.row0 + (2 * at.qt + s) * slot_tokens, &bar.q_full);
          ++items;
        }
      }
      items = __shfl_sync(0xffffffffu, items, 0);
      ok = __shfl_sync(0xffffffffu, (int)ok, 0);
      if (!ok) break;
      paged_from = 0x7fffffff;
      load(0, at.tile, tiles);
      for (int j = 0; ok && j < count; ++j) {
        load(1, at.tile + j, tiles + j);
        if (ok && j + 1 < count) load(0, at.tile + j + 1, tiles + j + 1);
      }
      tiles += count;
    }
    // every copy has landed before the block lets go of its shared memory
    if (lane == 0) {
      for (int k = max(0, n - BUFS); k < n; ++k) mbar_wait_drain(&full[k % BUFS], (uint32_t)(k / BUFS & 1));
      if (items > 0) mbar_wait_drain(&bar.q_full, (uint32_t)((items - 1) & 1));
    }
  } else if (warp == 9) {
    // ------------------------------------------------------- products --
    give_registers<C>();
    if (lane == 0) {
      constexpr uint32_t idS = idesc_bf16_f32(128, kKeys);
      constexpr uint32_t idO = idesc_bf16_f32(128, HD) | (1u << 16);  // B is MN-major
      int c = 0, items = 0, tiles = 0;
      uint32_t cleaned = 0;  // parity of each buffer's `ready` barrier (bf16: V only uses it)
      bool ok = true;
      auto wait = [&](uint64_t* b, uint32_t parity, int code) {
        return mbar_wait_bounded(b, parity, err, code, limit);
      };
      auto wait_k = [&](int c) {
        if (B16) return wait(&bar.full[c % C::RING], c / C::RING & 1, DEV_TIMEOUT_FULL);
        return wait(&bar.ready[c % C::RING], c / C::RING & 1, DEV_TIMEOUT_FULL);
      };
      auto issue_s = [&](int s, int buf) {
        const uint32_t q = smem_u32(sQ + s * C::BUF), k = smem_u32(ring + buf * C::BUF);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint32_t off = (ks >> 2) * (128 * 128);
          tc_mma_bf16(tmem + 128u * s, smem_desc_sw128(q + off) + 2 * (ks & 3), smem_desc_sw128(k + off) + 2 * (ks & 3),
                      idS, ks > 0 ? 1u : 0u);
        }
        tc_commit(&bar.s_full[s]);
      };
      auto issue_pv = [&](int s, int buf, bool first) {
        const uint32_t v = smem_u32(ring + buf * C::BUF);
#pragma unroll
        for (int ks = 0; ks < kKeys / 16; ++ks)
          tc_mma_ts(tmem + 256u + 128u * s, tmem + 128u * s + 8u * ks, smem_desc_mn_sw128(v, kKeys * 128) + 128 * ks, idO,
                    first && ks == 0 ? 0u : 1u);
      };
      for (bool next = true; ok && next; next = plan_next_item(a.plan, p, range, at)) {
        const int count = plan_here(range, at);
        if (count == 0) continue;
        ok = wait(&bar.q_full, items & 1, DEV_TIMEOUT_FULL) &&
             wait_k(c);
        if (!ok) break;
        tc_fence_after();
        issue_s(0, c % C::RING);
        issue_s(1, c % C::RING);
        tc_commit(&bar.empty[c % C::RING]);
        if (count == 1) tc_commit(&bar.q_empty);
        ++c;
        for (int j = 0; ok && j < count; ++j) {
          const int vb = c % C::RING, kb = (c + 1) % C::RING;
          const bool more = j + 1 < count;
          // landed, and clean
          ok = wait(&bar.ready[vb], B16 ? cleaned >> vb & 1u : c / C::RING & 1u, DEV_TIMEOUT_FULL);
          cleaned ^= 1u << vb;
          // O of the previous item has been read
          if (j == 0 && items > 0) ok = ok && wait(&bar.epilogue, (items - 1) & 1, DEV_TIMEOUT_ACC_EMPTY);
          ok = ok && wait(&bar.p_ready[0], (tiles + j) & 1, DEV_TIMEOUT_ACC_FULL);
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, vb, j == 0);
          if (more) {
            ok = wait_k(c + 1);
            if (!ok) break;
            tc_fence_after();
            issue_s(0, kb);
          } else {
            tc_commit(&bar.o_full[0]);
          }
          ok = wait(&bar.p_ready[1], (tiles + j) & 1, DEV_TIMEOUT_ACC_FULL);
          if (!ok) break;
          tc_fence_after();
          issue_pv(1, vb, j == 0);
          tc_commit(&bar.empty[vb]);
          if (more) {
            issue_s(1, kb);
            tc_commit(&bar.empty[kb]);
            if (j + 2 == count) tc_commit(&bar.q_empty);
          } else {
            tc_commit(&bar.o_full[1]);
          }
          c += more ? 2 : 1;
        }
        tiles += count;
        ++items;
      }
      // every product issued above has ended before tensor memory is freed
      tc_commit(&bar.drain);
      mbar_wait_drain(&bar.drain, 0);
    }
  } else if (warp >= C::CLEAN_WARP) {
    // -------------------------------------------- cleaning, expanding --
    give_registers<C>();
    // V tiles that not every row sees: slots that no row sees (past the
    // context, without a page) become zeros, and what is not finite among the
    // keys that only some rows see is noted and taken out -- a weight of 0
    // would not keep it out of the product.
    const int t = tid - 32 * C::CLEAN_WARP;
    int c = 0, items = 0, tiles = 0;
    bool ok = true;
    int seen_min = 0, seen_max = 0;
    // the previous item's notes have been read and cleared
    auto notes_free = [&]() {
      return mbar_wait_bounded(&bar.epilogue, notes_phase(items) & 1, err, DEV_TIMEOUT_ACC_EMPTY, limit);
    };
    // the row of one key of the V tile at k0 in buffer b
    auto clean_key = [&](int b, int k0, int key, uint32_t have) {
      const bool unseen = k0 + key >= seen_max || !(have >> (key >> 4) & 1u);
      if (!unseen && k0 + key < seen_min) return;  // all rows see it
      uint8_t* row = ring + b * C::BUF + key * 128;
      // piece i of the row, 16 bytes (as swizzled, i ^ key: any order will do to look)
      auto piece_at = [&](int i) {
        return reinterpret_cast<uint4*>(row + (i >> 3) * (kKeys * 128) + ((i & 7) << 4));
      };
      if (unseen) {
#pragma unroll
        for (int i = 0; i < HD / 8; ++i) *piece_at(i) = make_uint4(0, 0, 0, 0);
        return;
      }
      uint32_t odd = 0;  // bit i: piece i has an exponent of all ones
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        const uint4 x = *piece_at(i);
        const uint32_t carry = ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                               ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
        odd |= (carry & 0x80008000u) ? 1u << i : 0u;
      }
      if (odd == 0) return;
      if (items > 0) notes_free();
      bar.any_bad = 1;
      for (; odd != 0; odd &= odd - 1) {
        const int i = __ffs((int)odd) - 1;
        const int col = (i >> 3) * 64 + ((i ^ key) & 7) * 8;
        uint16_t* x = reinterpret_cast<uint16_t*>(piece_at(i));
        for (int e = 0; e < 8; ++e) {
          const uint32_t y = x[e];
          if ((y & 0x7f80u) != 0x7f80u) continue;
          Poison& n = bad[col + e];
          atomicMin((y & 0x7fu) ? &n.nan : (y & 0x8000u) ? &n.neg : &n.pos, k0 + key);
          x[e] = 0;
        }
      }
    };
    // tile `tile` of V (count-th of the block) in buffer b, as bf16
    auto clean = [&](int b, int tile, int count) {
      const int k0 = tile * kKeys;
      const uint32_t have = bar.with_page[count % 16];
      if (k0 + kKeys <= seen_min && have == 255u) return;
      for (int key = t; key < kKeys; key += 32 * C::CLEAN_WARPS) clean_key(b, k0, key, have);
    };
    // the next buffer of codes into the next bf16 buffer
    auto expand = [&]() {
      const int rb = c % C::RAW, b = c % C::RING;
      ok = mbar_wait_bounded(&bar.raw_full[rb], c / C::RAW & 1, err, DEV_TIMEOUT_FULL, limit) &&
           (c < C::RING || mbar_wait_bounded(&bar.empty[b], (c / C::RING - 1) & 1, err, DEV_TIMEOUT_EMPTY, limit));
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) return;
      constexpr int PIECES = HD / 16;  // of codes in a row
      const uint8_t* scales = raw + C::RAW * C::CODES + rb * kKeys;
#pragma unroll 1
      for (int i = t; i < kKeys * PIECES; i += 32 * C::CLEAN_WARPS) {
        const int key = i / PIECES, slot = i % PIECES;  // in the order they lie, so that no bank is met twice
        const int piece = HD == 128 ? slot ^ (key & 7) : slot ^ (key >> 1 & 3);
        const uint4 w = *reinterpret_cast<const uint4*>(raw + rb * C::CODES + 16 * i);
        const float scale = scale_of(scales[key]);
        const float2 scale2 = make_float2(scale, scale);
        const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
        uint32_t o[8];
#pragma unroll
        for (int h = 0; h < 8; ++h) {
          const __half2_raw x = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(ww[h >> 1] >> (16 * (h & 1))), __NV_E4M3);
          const float2 f = __fmul2_rn(__half22float2(__half2(x)), scale2);
          o[h] = pack_bf16x2(f.x, f.y);
        }
        uint8_t* row = ring + b * C::BUF + (piece >> 2) * (kKeys * 128) + key * 128;
        *reinterpret_cast<uint4*>(row + (((2 * piece & 7) ^ (key & 7)) << 4)) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(row + (((2 * piece + 1 & 7) ^ (key & 7)) << 4)) = make_uint4(o[4], o[5], o[6], o[7]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.raw_empty[rb]);
    };
    // Whether every warp's step went well: they go on, or stop, together.  (A
    // key's row is expanded by several threads, so they also have to meet.)
    auto agree = [&](bool mine) {
      uint32_t all;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 2, %2, p;\n\t"
          "selp.u32 %0, 1, 0, q;\n\t}"
          : "=r"(all)
          : "r"((uint32_t)mine), "n"(32 * C::CLEAN_WARPS)
          : "memory");
      return all != 0;
    };
    auto hand_over = [&](int b) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ready[b]);
    };
    for (bool more = true; ok && more; more = plan_next_item(a.plan, p, range, at)) {
      const int count = plan_here(range, at);
      if (count == 0) continue;
      const int rows = at.n * a.plan.group;
      seen_min = plan_visible(at, (long long)at.qt * 2 * slot_tokens);
      seen_max = plan_visible(at, (min((long long)rows, (at.qt + 1ll) * a.plan.rows) - 1) / a.plan.group);
      for (int j = 0; ok && j < count; ++j) {
        // K_0, then V_j, K_(j+1); every V tile passes here, so that these warps cannot fall behind the ring
        for (int pool = j == 0 ? 0 : 1; ok && pool < 3; ++pool) {
          const bool k = pool != 1;
          if (pool == 2 && j + 1 == count) break;
          const int b = c % C::RING;
          if constexpr (B16) {
            if (!k) {
              ok = mbar_wait_bounded(&bar.full[b], c / C::RING & 1, err, DEV_TIMEOUT_FULL, limit) &&
                   (!notes_hold_back(items, j, count) || notes_free());
              ok = __all_sync(0xffffffffu, ok);
              if (!ok) break;
              clean(b, at.tile + j, tiles + j);
              hand_over(b);
            }
          } else {
            expand();
            ok = agree(ok);
            if (!ok) break;
            if (!k && notes_hold_back(items, j, count)) {  // (in the meeting above: 232 us for 224, 32 x 10 rows)
              ok = notes_free();
              __syncwarp();
              ok = agree(ok);
              if (!ok) break;
            }
            if (!k) clean(b, at.tile + j, tiles + j);
            hand_over(b);
          }
          ++c;
        }
      }
      tiles += count;
      ++items;
    }
  } else {
    // -------------------------------------------------------- softmax --
    take_registers<C>();
    const int s = warp >> 2, r = tid & 127;  // slot, row of its tile = TMEM lane
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128u * s + lanes, tO = tmem + 256u + 128u * s + lanes;
    int tiles = 0, items = 0;
    for (bool more = true; more; more = plan_next_item(a.plan, p, range, at)) {
      const int count = plan_here(range, at);
      const bool whole = at.tile == 0 && count == at.tiles;
      const long long tok = (2ll * at.qt + s) * slot_tokens + r / a.plan.group;
      const bool valid = r < slot_tokens * a.plan.group && tok < at.n;
      const int visible = valid ? plan_visible(at, tok) : 0;
      const long long part =
          ((long long)blockIdx.x * 2 + (at.tile == 0 ? 1 : 0)) * a.plan.rows + (s * slot_tokens * a.plan.group + r);
      if (count == 0) {
        if (valid) {
          a.part_ml[part] = make_float2(-INFINITY, 0.f);
          for (int i = 0; i < HD; i += 4)
            *reinterpret_cast<float4*>(a.part + part * HD + i) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        continue;
      }
      const int seen_min = plan_visible(at, (long long)at.qt * 2 * slot_tokens);
      float m = -INFINITY, l = 0.f;
      // a warp whose wait gives up keeps to the loops; later waits give up at once
      bool ok = true;
      for (int j = 0; j < count; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait_bounded(&bar.s_full[s], (tiles + j) & 1, err, DEV_TIMEOUT_ACC_FULL, limit));
        if (ok) {
          tc_fence_after();
          const int k0 = (at.tile + j) * kKeys;
          const uint32_t have = bar.with_page[(tiles + j) % 16];
          const bool masked = k0 + kKeys > seen_min || have != 255u;
          // keys of chunk q that this row sees, as bits
          auto sees = [&](int q) {
            const int n = visible - k0 - 32 * q;
            const uint32_t low = n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
            return low & ((have >> (2 * q) & 1u) * 0xffffu | (have >> (2 * q + 1) & 1u) * 0xffff0000u);
          };
          auto mask_chunk = [&](int q, uint32_t* x) {
            const uint32_t bits = sees(q);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(bits >> i & 1u)) x[i] = 0xff800000u;  // -inf
          };
          auto max_chunk = [&](const uint32_t* x, float* mx) {
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              mx[i >> 1 & 1] = fmaxf(mx[i >> 1 & 1], fmaxf(__uint_as_float(x[i]), __uint_as_float(x[i + 1])));
          };
          uint32_t w[64];  // the weights, two bf16 each
          float2 sum[2];
          float mx[2];
          // weights of the tile against reference `ref`, 32 scores at a time
          // with the next 32 on their way; the scores' maximum goes along
          auto weigh = [&](float ref, auto with_mask) {
            const float2 c2 = make_float2(a.scale_log2, a.scale_log2), n2 = make_float2(-ref, -ref);
            sum[0] = sum[1] = make_float2(0.f, 0.f);
            mx[0] = mx[1] = -INFINITY;
            uint32_t x[2][32];
            tmem_ld32_async(tS, x[0]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t* y = x[q & 1];
              tmem_wait_ld();
              if (q < 3) tmem_ld32_async(tS + 32 * (q + 1), x[(q + 1) & 1]);
              if constexpr (with_mask()) mask_chunk(q, y);
              max_chunk(y, mx);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 z = __ffma2_rn(make_float2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), c2, n2);
                const float2 e = make_float2(fast_exp2(z.x), fast_exp2(z.y));
                sum[i >> 1 & 1] = __fadd2_rn(sum[i >> 1 & 1], e);
                w[16 * q + (i >> 1)] = pack_bf16x2(e.x, e.y);
              }
            }
          };
          // Most tiles leave the reference as it is: weigh against it at once
          // and look afterwards whether that held.
          bool settled = false;
          if (!masked && !__any_sync(0xffffffffu, m == -INFINITY)) {
            weigh(m, std::false_type());
            settled = !__any_sync(0xffffffffu, fmaxf(mx[0], mx[1]) * a.scale_log2 > m + 8.f);
          }
          if (!settled) {
            mx[0] = mx[1] = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < 4; ++q) {
              uint32_t x[32];
              tmem_ld32_async(tS + 32 * q, x);
              tmem_wait_ld();
              if (masked) mask_chunk(q, x);
              max_chunk(x, mx);
            }
            const float top = fmaxf(mx[0], mx[1]) * a.scale_log2;
            const bool raise = top > m + 8.f || (m == -INFINITY && top > -INFINITY);
            if (__any_sync(0xffffffffu, raise)) {
              const float corr = raise ? fast_exp2(m - top) : 1.f;  // 0 for the first
              if (raise) m = top;
              l *= corr;
              if (j > 0) {
#pragma unroll 1
                for (int q = 0; q < HD / 32; ++q) {
                  uint32_t o[32];
                  tmem_ld32_async(tO + 32 * q, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
                  tmem_st32(tO + 32 * q, o);
                }
              }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            if (masked)
              weigh(ref, std::true_type());
            else
              weigh(ref, std::false_type());
          }
          tmem_st32(tS, w);  // over the scores, which have all been used
          tmem_st32(tS + 32, w + 32);
          l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_ready[s]);
      }
      const bool got = __all_sync(
          0xffffffffu, mbar_wait_bounded(&bar.o_full[s], items & 1, err, DEV_TIMEOUT_ACC_FULL, limit));
      if (got && ok) {
        tc_fence_after();
        const bool poisoned = bar.any_bad != 0;
        // weight_share of the seen reference, in the form that spills least: 2 x
        // 1,024 rows over bf16 475 us for 480, over codes with head_dim 64 486 for 506
        float inv;
        if constexpr (B16) {
          m = seen_reference(m, bar.paged_from[items % 4] < visible);
          inv = weight_share(l, m);
        } else {
          if (l == 0.f) m = seen_reference(m, bar.paged_from[items % 4] < visible);
          inv = l == 0.f ? (m == -INFINITY ? 0.f : NAN) : __fdividef(1.f, l);  // (2^-22 off)
        }
        bf16* dst = a.out + (long long)(at.row0 + tok) * a.out_stride +
                    (at.head * a.plan.group + r % a.plan.group) * HD;
#pragma unroll 1
        for (int q = 0; q < HD / 32; ++q) {
          uint32_t x[32];
          tmem_ld32_async(tO + 32 * q, x);
          tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            o[i] = __uint_as_float(x[i]);
            if (poisoned) o[i] += poison_of(bad[32 * q + i], visible);
          }
          if (!valid) continue;
          if (whole) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 y;
              y.x = pack_bf16x2(o[i] * inv, o[i + 1] * inv);
              y.y = pack_bf16x2(o[i + 2] * inv, o[i + 3] * inv);
              y.z = pack_bf16x2(o[i + 4] * inv, o[i + 5] * inv);
              y.w = pack_bf16x2(o[i + 6] * inv, o[i + 7] * inv);
              *reinterpret_cast<uint4*>(dst + 32 * q + i) = y;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(a.part + part * HD + 32 * q + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        if (valid && !whole) a.part_ml[part] = make_float2(m, l);
        tc_fence_before();
      }
      // every softmax warp has read the notes before they are cleared for the next item
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (bar.any_bad != 0) {
        for (int i = tid; i < HD; i += kSoftmaxThreads) bad[i] = Poison{0x7fffffff, 0x7fffffff, 0x7fffffff};
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (tid == 0) bar.any_bad = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.epilogue);
      tiles += count;
      ++items;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Tensor map of the queries: [row][head][head_dim], boxes of one slot's
// tokens of a kv head's group.
bool encode_queries(CUtensorMap* map, const PagedArgs& a, int n_rows, int n_q_heads, int hd, int slot_tokens) {
  const cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)n_q_heads, (cuuint64_t)n_rows};
  const cuuint64_t strides[2] = {(cuuint64_t)hd * 2, (cuuint64_t)a.q_stride * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)a.plan.group, (cuuint32_t)slot_tokens};
  return encode_tmap_tiled3(map, a.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int HD, int TYPE>
armt_status launch(const PagedArgs& a, const PagedView& p, const armt_kv_cache& cache, int n_q_heads, cudaStream_t st) {
  using C = TileCfg<HD, TYPE>;
  static DeviceOnce once;
  if (once.need(a.device)) {
    cudaError_t e =
        cudaFuncSetAttribute(tiles_kernel<HD, TYPE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    cudaFuncAttributes at;
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&at, tiles_kernel<HD, TYPE>);
    if (e != cudaSuccess) return launch_status(e, "paged attention set-up");
    if (!C::B16 && !split_fits(at.numRegs, C::THREADS, kSoftmaxThreads, C::SOFTMAX_REGS, C::OTHER_REGS))
      return refuse(ARMT_ERR_CUDA, "paged attention: unexpected register count");
    once.set(a.device);
  }
  const int slot_tokens = 128 / a.plan.group;
  CUtensorMap tm_q, tm_k, tm_v;
  if (!encode_pool(&tm_k, p.k, cache, kKeys) || !encode_pool(&tm_v, p.v, cache, kKeys) ||
      !encode_queries(&tm_q, a, p.n_rows, n_q_heads, HD, slot_tokens))
    return refuse(ARMT_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  tiles_kernel<HD, TYPE><<<a.plan.blocks, C::THREADS, C::SMEM, st>>>(tm_q, tm_k, tm_v, a, p, slot_tokens);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_join(a, p, HD, false, st);
  return launch_status(e, "paged attention");
}

}  // namespace

int tile_rows(int group) { return 2 * (128 / group) * group; }

armt_status launch_tiles(const PagedArgs& args, const PagedView& p, const armt_kv_cache& cache, int n_q_heads,
                         cudaStream_t st) {
  static DeviceSymbol word;
  PagedArgs a = args;
  const cudaError_t e = word.find(g_tiles_err, a.device, &a.own_err);
  if (e != cudaSuccess) return launch_status(e, "paged attention set-up");
  a.plan.keys = kKeys;
  a.plan.fixed = 5 * kKeys;  // an item's beginning and end take about as long as five tiles
  a.plan.least = 2;
  if (cache.type == ARMT_CACHE_BF16)
    return cache.head_dim == 64 ? launch<64, ARMT_CACHE_BF16>(a, p, cache, n_q_heads, st)
                                : launch<128, ARMT_CACHE_BF16>(a, p, cache, n_q_heads, st);
  return cache.head_dim == 64 ? launch<64, ARMT_CACHE_E4M3>(a, p, cache, n_q_heads, st)
                              : launch<128, ARMT_CACHE_E4M3>(a, p, cache, n_q_heads, st);
}

}  // namespace armt
