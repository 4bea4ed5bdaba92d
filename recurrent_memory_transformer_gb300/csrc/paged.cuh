// The paged key/value cache as the kernels see it, and the checks of its
// descriptors that the entry points share.
//
// Pools are [page][kv head][slot][head_dim], so one head's rows of a page are
// contiguous: a 16-token page of 128 bf16 is a 4 KB run for the attention's
// loads, and the rows of a prompt, written token after token, fill whole
// lines.  Nothing read from the batch's device arrays is trusted: a sequence
// or page that does not fit counts as empty.
#pragma once

#include <cuda_fp8.h>

#include <exception>
#include <new>
#include <string>

#include "../../include/armt.h"
#include "common.cuh"

namespace armt {

void set_last_error(const std::string& msg);       // text returned by armt_last_error()
armt_status ready_device(int* dev, int* num_sms);  // the current device, if the kernels run on it
armt_status block_error_word(int dev, int** word);  // what armt_block_sync_status reads and clears
void* current_context();

bool encode_tmap_tiled3(CUtensorMap* map, const void* base, CUtensorMapDataType type, const cuuint64_t* dims,
                        const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle);

inline armt_status refuse(armt_status s, const std::string& msg) {
  set_last_error(msg);
  return s;
}

// No exception leaves a C entry point.
template <typename F>
armt_status guarded(F body) noexcept {
  try {
    return body();
  } catch (const std::bad_alloc&) {
    return ARMT_ERR_OOM;
  } catch (const std::exception&) {
    return ARMT_ERR_CUDA;
  }
}

// One bit a device: whether its set-up of a kernel has been done.
struct DeviceOnce {
  std::atomic<unsigned long long> done{0};
  bool need(int dev) const { return dev < 0 || dev > 63 || !(done.load() >> dev & 1); }
  void set(int dev) {
    if (dev >= 0 && dev < 64) done.fetch_or(1ull << dev);
  }
};

inline armt_status launch_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return ARMT_OK;
  return refuse(ARMT_ERR_CUDA, std::string(what) + ": " + cudaGetErrorString(e));
}

struct PagedView {
  uint8_t *k, *v;              // pools
  uint8_t *k_scale, *v_scale;  // scale bytes (e4m3)
  const int32_t *row_start, *kv_len, *table;
  int n_pages, page_shift, hkv;
  int n_seqs, table_width, max_new;
  int n_rows;
};

// One sequence's rows: n new rows from row0 on (n as given; rows past the
// first max_new are left out by the callers), positions up to kv_len - 1.
struct PagedSeq {
  int row0, n, kv_len;
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedView& p, int b) {
  PagedSeq s;
  s.row0 = p.row_start[b];
  const int end = p.row_start[b + 1];
  s.kv_len = p.kv_len[b];
  s.n = (s.row0 < 0 || end > p.n_rows || end < s.row0) ? 0 : end - s.row0;
  return s;
}

// Page of position `pos` of sequence b, -1 if it has none.
__device__ __forceinline__ int paged_page(const PagedView& p, int b, long long pos) {
  if (pos < 0 || (pos >> p.page_shift) >= p.table_width) return -1;
  const int page = __ldg(p.table + (long long)b * p.table_width + (pos >> p.page_shift));
  return (unsigned)page < (unsigned)p.n_pages ? page : -1;
}

// Index of a row of one kv head: (page * hkv + head) * page_size + slot.
__device__ __forceinline__ long long paged_row(const PagedView& p, int page, int head, int slot) {
  return ((((long long)page * p.hkv + head) << p.page_shift) + slot);
}

// 2^(byte - 127): the byte is the exponent field of an fp32.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// ------------------------------------------------------------- checks --

inline bool misaligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

inline armt_status check_cache(const armt_kv_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return refuse(ARMT_ERR_ARG, "NULL argument");
  if (c->type != ARMT_CACHE_BF16 && c->type != ARMT_CACHE_E4M3) return refuse(ARMT_ERR_ARG, "bad cache type");
  if (c->type == ARMT_CACHE_E4M3 && (c->k_scale == nullptr || c->v_scale == nullptr))
    return refuse(ARMT_ERR_ARG, "an e4m3 cache needs k_scale and v_scale");
  if (c->n_pages <= 0 || c->n_kv_heads <= 0) return refuse(ARMT_ERR_ARG, "sizes must be positive");
  if (c->n_pages > 0x7fffffffll) return refuse(ARMT_ERR_SHAPE, "n_pages must be at most 2^31 - 1");
  if (c->n_pages * c->n_kv_heads > 0x7fffffffll)
    return refuse(ARMT_ERR_SHAPE, "n_pages * n_kv_heads must be at most 2^31 - 1");
  if (c->n_kv_heads > 1024) return refuse(ARMT_ERR_SHAPE, "n_kv_heads must be at most 1024");
  if (c->head_dim != 64 && c->head_dim != 128)
    return refuse(ARMT_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return refuse(ARMT_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
  if (misaligned16(c->k) || misaligned16(c->v) ||
      (c->type == ARMT_CACHE_E4M3 && (misaligned16(c->k_scale) || misaligned16(c->v_scale))))
    return refuse(ARMT_ERR_ARG, "pointers must be 16-byte aligned");
  return ARMT_OK;
}

inline armt_status check_batch(const armt_paged_batch* b, const armt_kv_cache* c) {
  if (b == nullptr || b->row_start == nullptr || b->kv_len == nullptr || b->page_table == nullptr)
    return refuse(ARMT_ERR_ARG, "NULL argument");
  if ((reinterpret_cast<uintptr_t>(b->row_start) | reinterpret_cast<uintptr_t>(b->kv_len) |
       reinterpret_cast<uintptr_t>(b->page_table)) & 3)
    return refuse(ARMT_ERR_ARG, "row_start, kv_len and page_table must be 4-byte aligned");
  if (b->n_seqs <= 0 || b->table_width <= 0 || b->max_new <= 0 || b->n_rows < 0)
    return refuse(ARMT_ERR_ARG, "sizes must be positive");
  if (b->n_seqs > 65535) return refuse(ARMT_ERR_SHAPE, "n_seqs must be at most 65535");
  if (b->n_rows > 0x7fffffffll) return refuse(ARMT_ERR_SHAPE, "n_rows must be at most 2^31 - 1");
  if ((int64_t)b->table_width * c->page_size > (1ll << 30))
    return refuse(ARMT_ERR_SHAPE, "table_width * page_size must be at most 2^30");
  return ARMT_OK;
}

// n rows `stride` elements apart, `width` elements used of each.
inline armt_status check_rows(const void* p, int64_t n, int64_t stride, int64_t width, const char* name) {
  if (p == nullptr && n > 0) return refuse(ARMT_ERR_ARG, "NULL argument");
  if (misaligned16(p)) return refuse(ARMT_ERR_ARG, "pointers must be 16-byte aligned");
  if (stride < width || stride % 8 != 0 || stride > (1ll << 31))
    return refuse(ARMT_ERR_SHAPE, std::string(name) + ": a row stride must be a multiple of 8, at least " +
                                      std::to_string(width) + " and at most 2^31");
  return ARMT_OK;
}

inline PagedView paged_view(const armt_kv_cache& c, const armt_paged_batch& b) {
  PagedView v;
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.row_start = b.row_start;
  v.kv_len = b.kv_len;
  v.table = b.page_table;
  v.n_pages = (int)c.n_pages;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c.page_size) ++v.page_shift;
  v.hkv = c.n_kv_heads;
  v.n_seqs = b.n_seqs;
  v.table_width = b.table_width;
  v.max_new = b.max_new;
  v.n_rows = (int)b.n_rows;
  return v;
}

}  // namespace armt
