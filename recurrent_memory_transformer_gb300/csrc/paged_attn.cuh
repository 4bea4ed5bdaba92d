// What the paged attention's two kernels share: arguments, tensor maps of the
// pools, the bookkeeping of non-finite values, and the joining kernel's launch.
#pragma once

#include "paged_plan.cuh"

namespace armt {

struct PagedArgs {
  const bf16* q;
  bf16* out;
  long long q_stride, out_stride;
  float scale_log2;
  PagedPlan plan;
  float* part;  // [block][2][plan.rows][head_dim], then the (reference, sum) of each row,
  float2* part_ml;  // or (reference, the sum's reference, sum, -) from the few-row kernels over codes
  PlanRange* plans;  // [block]: what each block found for itself, for the joining kernel
  WaitPolicy wp;
  int device;
  int* own_err;  // the kernel's own error word, and the building blocks', which
  int* err;      // armt_block_sync_status reads: the joining kernel passes one on to the other
};

// A device global's address on each device, looked up when the device's context is
// new (and without device work, which a capture would refuse).
struct DeviceSymbol {
  std::atomic<void*> ctx[64] = {};
  std::atomic<int*> at[64] = {};
  cudaError_t find(const int& symbol, int dev, int** out) {
    if (dev < 0 || dev > 63) return cudaErrorInvalidDevice;
    void* now = current_context();
    *out = at[dev].load();
    if (*out != nullptr && ctx[dev].load() == now) return cudaSuccess;
    void* p = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&p, symbol);
    if (e != cudaSuccess) return e;
    *out = static_cast<int*>(p);
    at[dev].store(*out);
    ctx[dev].store(now);
    return cudaSuccess;
  }
};

// Untiled copy of n bytes (a multiple of 16, both ends 16-byte aligned).
__device__ __forceinline__ void bulk_load(void* dst, const void* src, int n, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(n), "r"(smem_u32(bar))
               : "memory");
}
// The calling block's range, in shared memory, and kept for the joining kernel.
__device__ __forceinline__ void plan_and_keep(const PagedArgs& a, const PagedView& p, PlanScratch& s, PlanRange& r) {
  plan_range(a.plan, p, (int)blockIdx.x, s, r);
  if (threadIdx.x == 0) a.plans[blockIdx.x] = r;
}

// Where non-finite values sit in a head's value columns among keys that only
// some of a tile's rows may see.  0 * NaN is NaN, so such values are taken out
// of the product and what they do to the rows that do see them is added at
// the end: for each column the first key with NaN, +inf and -inf.
struct Poison {
  int nan, pos, neg;
};

__device__ __forceinline__ float poison_of(const Poison& t, int visible) {
  float v = 0.f;
  if (t.pos < visible) v += INFINITY;
  if (t.neg < visible) v -= INFINITY;  // NaN with both
  if (t.nan < visible) v = NAN;
  return v;
}

// Rows without weights.  One that attends to nothing gives zeros; one that
// attends to keys whose scores are all -inf is 0 / 0 in the softmax and gives NaN.
// The second kind leaves the loops with the reference -inf like the first, and
// takes the lowest number for it instead, which says so to the joining kernel too
// and weighs nothing beside any part with weights.
__device__ __forceinline__ float seen_reference(float m, bool sees_a_key) {
  return m == -INFINITY && sees_a_key ? -3.402823466e38f : m;
}
// 1 / (sum of weights), or what stands for it in such rows.
__device__ __forceinline__ float weight_share(float l, float m) {
  return l != 0.f ? 1.f / l : m == -INFINITY ? 0.f : NAN;
}

// Tensor map of a pool: rows of head_dim elements, page_size of them, a page
// of one head after another; boxes of the rows that a tile of `keys` has in
// one page, 128 bytes (64 for 64-byte rows) wide and swizzled over that width.
inline bool encode_pool(CUtensorMap* map, const void* pool, const armt_kv_cache& c, int keys) {
  const bool b16 = c.type == ARMT_CACHE_BF16;
  const cuuint32_t width = b16 || c.head_dim == 64 ? 64 : 128;
  const cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.page_size,
                              (cuuint64_t)c.n_pages * (cuuint64_t)c.n_kv_heads};
  const cuuint64_t row = (cuuint64_t)c.head_dim * (b16 ? 2 : 1);
  const cuuint64_t strides[2] = {row, row * (cuuint64_t)c.page_size};
  const cuuint32_t box[3] = {width, (cuuint32_t)(c.page_size < keys ? c.page_size : keys), 1};
  return encode_tmap_tiled3(map, pool, b16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, dims,
                            strides, box,
                            !b16 && c.head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Launches the kernel that adds up the parts, as the dependent of the kernel
// launched before it on the stream (which lets it in early).  `two`: the parts
// have two references.
cudaError_t launch_join(const PagedArgs& a, const PagedView& p, int head_dim, bool two, cudaStream_t st);

// The tensor-core kernel for many query rows (paged_tiles.cu): its query
// tile's rows for a group of `group` heads, and its launch.
int tile_rows(int group);
armt_status launch_tiles(const PagedArgs& a, const PagedView& p, const armt_kv_cache& cache, int n_q_heads,
                         cudaStream_t st);

}  // namespace armt
