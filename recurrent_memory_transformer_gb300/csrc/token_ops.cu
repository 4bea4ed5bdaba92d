// From logits rows to tokens: probabilities, and the check of drafted tokens.
//
// Both walk rows of the vocabulary once, so HBM bounds them for a batch and
// the latency of a few dependent steps for one user.  A row is split over a
// thread-block cluster, so that five rows of 128,256 still use many SMs, and
// the CTAs of a row exchange one (maximum, sum) or one sum through distributed
// shared memory: each pushes its own to every peer (once all have
// started) and one cluster barrier later reads its local copies, so no CTA has
// to wait for its peers to exit.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace cg = cooperative_groups;
using namespace armt;

namespace {

constexpr int kMaxCluster = 8;  // the portable limit

// First half of a cluster barrier, and its second.  Every CTA arrives as it
// starts and waits before it writes into a peer, which has then started too.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// -------------------------------------------------------- probabilities --
//
// p = 2^((x - m) c) / sum, c = log2(e) / t.  Each CTA takes its slice of the
// row into registers (RV groups of 4 values a thread), works with the slice's
// own maximum m_c, and after the exchange scales by 2^((m_c - M) c) / S: one
// read and one write of the row.  All in fp32; the exponentials are the hardware's
// ex2 (2^-22), twice a value: 6e-8 to 2.2e-7 against 64 bits, a plain fp32 softmax
// 3e-8 to 1e-7.

constexpr int kProbThreads = 512;
struct RowPart {
  float m, s;
  int at;  // greedy rows: first index of the slice's maximum
};

// One group of 4 values: consecutive ones where rows are 16-byte aligned, a
// thread block's width apart otherwise (coalesced either way).
template <bool VEC>
__device__ __forceinline__ int elem_index(int j, int i) {
  return VEC ? 4 * ((int)threadIdx.x + kProbThreads * j) + i : (int)threadIdx.x + kProbThreads * (4 * j + i);
}

template <bool VEC>
__device__ __forceinline__ void load4(const float* src, int n, int j, float* v) {
  if (VEC && elem_index<VEC>(j, 3) < n) {
    const float4 x = __ldcs(reinterpret_cast<const float4*>(src + elem_index<VEC>(j, 0)));
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = elem_index<VEC>(j, i) < n ? __ldcs(src + elem_index<VEC>(j, i)) : -INFINITY;
  }
}

template <bool VEC>
__device__ __forceinline__ void store4(float* dst, int n, int j, const float* v) {
  if (VEC && elem_index<VEC>(j, 3) < n) {
    __stcs(reinterpret_cast<float4*>(dst + elem_index<VEC>(j, 0)), make_float4(v[0], v[1], v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (elem_index<VEC>(j, i) < n) __stcs(dst + elem_index<VEC>(j, i), v[i]);
  }
}

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & (kProbThreads / 32 - 1)];
#pragma unroll
  for (int o = kProbThreads / 64; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// RV > 0: a slice is at most 4 RV values a thread and stays in registers;
// RV = 0 (rows past 8 x 16,384): the slice is walked twice.
template <bool VEC, int RV>
__global__ void __launch_bounds__(kProbThreads) token_probs_kernel(const float* logits, long long ld_logits,
                                                                  const float* __restrict__ temperature, int vocab,
                                                                  int slice, float* probs, long long ld_probs,
                                                                  int clusters) {
  __shared__ float red_m[kProbThreads / 32], red_s[kProbThreads / 32];
  __shared__ int red_at;
  __shared__ RowPart parts[kMaxCluster];
  const cg::cluster_group cl = cg::this_cluster();
  if (clusters > 1) cluster_arrive();
  const int rank = (int)(blockIdx.x % (unsigned)clusters);
  const long long row = blockIdx.x / (unsigned)clusters;
  const int first = min(rank * slice, vocab), n = min(slice, vocab - first);
  const float* src = logits + row * ld_logits + first;
  float* dst = probs + row * ld_probs + first;
  const float t = temperature ? __ldg(temperature + row) : 1.f;
  const bool greedy = t <= 0.f;
  float c = 1.4426950408889634f / t;
  if (c > 3.0e38f) c = 3.0e38f;  // a tiny t: 0 * c stays 0 (and a NaN stays NaN)
  constexpr int HELD = RV > 0 ? RV : 1;
  float x[HELD][4];
  float m = -INFINITY;
  const int rounds = RV > 0 ? RV : (n + 4 * kProbThreads - 1) / (4 * kProbThreads);
  if (threadIdx.x == 0) red_at = 0x7fffffff;
#pragma unroll
  for (int j = 0; j < (RV > 0 ? RV : rounds); ++j) {
    float* v = x[RV > 0 ? j : 0];
    load4<VEC>(src, n, j, v);
    if (RV == 0) m = fmaxf(fmaxf(m, fmaxf(v[0], v[1])), fmaxf(v[2], v[3]));
  }
  if (RV > 0) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) m = fmaxf(fmaxf(m, fmaxf(x[j][0], x[j][1])), fmaxf(x[j][2], x[j][3]));
  }
  m = block_max(m, red_m);
  const float ref = m == -INFINITY ? 0.f : m;
  float s = 0.f;
  int at = 0x7fffffff;
#pragma unroll
  for (int j = 0; j < (RV > 0 ? RV : rounds); ++j) {
    float* v = x[RV > 0 ? j : 0];
    if (RV == 0) load4<VEC>(src, n, j, v);
    if (greedy) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // a thread's elements come in rising order: keep the first
        const bool hit = at == 0x7fffffff && v[i] == m && elem_index<VEC>(j, i) < n;
        at = hit ? elem_index<VEC>(j, i) : at;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = fast_exp2((v[i] - ref) * c);
        s += v[i];
      }
    }
  }
  s = warp_sum(s);
  if (greedy) at = __reduce_min_sync(0xffffffffu, at);
  if ((threadIdx.x & 31) == 0) {
    red_s[threadIdx.x >> 5] = s;
    if (greedy) atomicMin(&red_at, at);
  }
  if (clusters > 1) cluster_wait();
  __syncthreads();
  if (threadIdx.x < 32) {
    s = (int)threadIdx.x < kProbThreads / 32 ? red_s[threadIdx.x] : 0.f;
    s = warp_sum(s);
    if ((int)threadIdx.x < clusters) {
      const RowPart mine{m, s, red_at == 0x7fffffff ? red_at : red_at + first};
      if (clusters > 1)
        *cl.map_shared_rank(&parts[rank], threadIdx.x) = mine;
      else
        parts[0] = mine;
    }
  }
  if (clusters > 1)
    cl.sync();
  else
    __syncthreads();
  float M = -INFINITY;
  for (int k = 0; k < clusters; ++k) M = fmaxf(M, parts[k].m);
  if (greedy) {
    int win = 0x7fffffff;
    if (M > -INFINITY)
      for (int k = 0; k < clusters; ++k)
        if (parts[k].m == M) win = min(win, parts[k].at);
    for (int j = 0; j < (n + 4 * kProbThreads - 1) / (4 * kProbThreads); ++j) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = first + elem_index<VEC>(j, i) == win ? 1.f : 0.f;
      store4<VEC>(dst, n, j, v);
    }
    return;
  }
  float S = 0.f;
  for (int k = 0; k < clusters; ++k) {
    const float f = parts[k].m == -INFINITY ? 1.f : fast_exp2((parts[k].m - M) * c);
    S += parts[k].s * f;
  }
  // all of the row is -inf: S = 0 and zeros come out
  const float scale = S == 0.f ? 0.f : (m == -INFINITY ? 1.f : fast_exp2((m - M) * c)) / S;
#pragma unroll
  for (int j = 0; j < (RV > 0 ? RV : rounds); ++j) {
    float* v = x[RV > 0 ? j : 0];
    if (RV == 0) {
      load4<VEC>(src, n, j, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = fast_exp2((v[i] - ref) * c);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] *= scale;
    store4<VEC>(dst, n, j, v);
  }
}

// --------------------------------------------------------- verification --
//
// Every CTA of a sequence's cluster finds the number of accepted drafts for
// itself (a few gathered values), then sums its slice of r = max(p - q, 0),
// which its warps hold in registers, each a contiguous part in rounds of 128
// values.  A lane keeps its running sum as an unevaluated pair of floats (the
// two-sum of Knuth, 6 additions: double additions run at 1/64 of the rate
// here), and the lanes' pairs are added the same way.  The drawn token is
// where the running sum passes u * total: found by CTA, then warp, then round,
// then lane, the last step in doubles.

struct Pair {
  float hi, lo;
};
__device__ __forceinline__ void add_exact(Pair& a, float x) {
  const float s = a.hi + x, bb = s - a.hi;
  a.lo += (a.hi - (s - bb)) + (x - bb);
  a.hi = s;
}
__device__ __forceinline__ Pair warp_sum_pair(Pair a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, a.hi, o), lo = __shfl_xor_sync(0xffffffffu, a.lo, o);
    add_exact(a, hi);
    a.lo += lo;
  }
  return a;
}

// Where the running sum of `n` values, one a lane, first passes `mark`: the
// lane, with *before the sum up to it; n if it never does (-1: all are zero),
// *before then being of no use.  For a whole warp; doubles are slow, so one
// warp of a block looks and tells the others.
__device__ __forceinline__ int passes_at(double value, int n, double mark, double* before) {
  const int lane = threadIdx.x & 31;
  double run = lane < n ? value : 0.0;
  const bool positive = run > 0.0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, run, o);
    if (o < n && lane >= o) run += y;
  }
  double prev = __shfl_up_sync(0xffffffffu, run, 1);
  if (lane == 0) prev = 0.0;
  const uint32_t any = __ballot_sync(0xffffffffu, positive);
  const uint32_t past = __ballot_sync(0xffffffffu, positive && run + *before > mark);
  if (any == 0) return -1;
  if (past == 0) return n;
  const int at = __ffs((int)past) - 1;
  *before += __shfl_sync(0xffffffffu, prev, at);
  return at;
}
__device__ __forceinline__ int last_positive(double value, int n) {
  const uint32_t any = __ballot_sync(0xffffffffu, (int)(threadIdx.x & 31) < n && value > 0.0);
  return any == 0 ? -1 : 31 - __clz((int)any);
}

struct Residual {
  const float *p, *q;  // target row; draft row or NULL
  int sure;            // the draft token that was certain (q NULL), or -1
  int vocab;
  bool vec;
  // r at v..v + 3 (zeros past the vocabulary)
  __device__ __forceinline__ void at4(int v, float* r) const {
    float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
    if (vec && v + 3 < vocab) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p + v));
      a[0] = x.x, a[1] = x.y, a[2] = x.z, a[3] = x.w;
      if (q) {
        const float4 y = __ldg(reinterpret_cast<const float4*>(q + v));
        b[0] = y.x, b[1] = y.y, b[2] = y.z, b[3] = y.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = v + i < vocab ? __ldg(p + v + i) : 0.f;
        if (q && v + i < vocab) b[i] = __ldg(q + v + i);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (v + i == sure) b[i] = 1.f;
      r[i] = fminf(fmaxf(a[i] - b[i], 0.f), 2.f);  // NaN gives 0
    }
  }
};

// RV > 0: a warp's part is at most RV rounds and stays in registers; RV = 0:
// the one warp that draws walks its part again out of L2, which leaves
// registers for more blocks on an SM.
template <int WARPS, int RV>
__global__ void __launch_bounds__(32 * WARPS) verify_drafts_kernel(
    const float* __restrict__ target, long long ld_target, const float* __restrict__ draft, long long ld_draft,
    const int32_t* __restrict__ tokens, const int32_t* __restrict__ start, const float* __restrict__ uniform,
    int n_drafts, int vocab, int rounds, bool vec, int32_t* n_accepted, int32_t* out_tokens, int clusters) {
  __shared__ int s_accepted;
  __shared__ double warp_part[WARPS];
  __shared__ double cta_part[2][kMaxCluster];
  __shared__ struct {
    double before, mark;
    int warp;
  } pick;
  const cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)(blockIdx.x % (unsigned)clusters), b = (int)(blockIdx.x / (unsigned)clusters);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d0 = start[b], d1 = start[b + 1];
  if (d0 < 0 || d1 < d0 || d1 > n_drafts) return;  // the whole cluster alike
  if (clusters > 1) cluster_arrive();
  const int n = d1 - d0;
  const long long row0 = (long long)d0 + b;
  const float u = uniform[row0 + n];
  if (threadIdx.x == 0) s_accepted = n;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 32 * WARPS) {
    const int x = tokens[d0 + i];
    const float ui = uniform[row0 + i];
    float p = 0.f, q = 1.f;
    if ((unsigned)x < (unsigned)vocab) {
      p = target[(row0 + i) * ld_target + x];
      if (draft) q = draft[(long long)(d0 + i) * ld_draft + x];
    }
    if (!(__fmul_rn(ui, q) < p)) {
      atomicMin(&s_accepted, i);
      break;
    }
  }
  __syncthreads();
  const int a = s_accepted;
  if (rank == 0) {
    if (threadIdx.x == 0) n_accepted[b] = a;
    for (int i = threadIdx.x; i <= n; i += 32 * WARPS)
      if (i != a) out_tokens[row0 + i] = i < a ? tokens[d0 + i] : -1;
  }
  Residual res;
  res.p = target + (row0 + a) * ld_target;
  res.q = a < n && draft ? draft + (long long)(d0 + a) * ld_draft : nullptr;
  res.sure = a < n && !draft ? tokens[d0 + a] : -1;
  res.vocab = vocab;
  res.vec = vec;
  // this warp's part: `rounds` rounds of 128 values, one after another
  const long long base = ((long long)rank * WARPS + warp) * rounds * 128 + 4 * lane;
  const int begin = (int)min(base, (long long)vocab);  // this lane's first value (vocab: none)
  constexpr int HELD = RV > 0 ? RV : 1;
  float r[HELD][4];
  for (int attempt = 0; attempt < 2; ++attempt) {
    Pair acc{0.f, 0.f};
    if constexpr (RV > 0) {
#pragma unroll
      for (int j = 0; j < RV; ++j) {
        r[j][0] = r[j][1] = r[j][2] = r[j][3] = 0.f;
        if (j < rounds && begin + 128ll * j < vocab) res.at4(begin + 128 * j, r[j]);
      }
    }
    if constexpr (RV > 0) {
#pragma unroll
      for (int j = 0; j < RV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) add_exact(acc, r[j][i]);
    } else {
      for (int j0 = 0; j0 < rounds; j0 += 4) {  // four rounds' loads at a time
        float x[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j][0] = x[j][1] = x[j][2] = x[j][3] = 0.f;
          if (j0 + j < rounds && begin + 128ll * (j0 + j) < vocab) res.at4(begin + 128 * (j0 + j), x[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) add_exact(acc, x[j][i]);
      }
    }
    acc = warp_sum_pair(acc);
    if (lane == 0) warp_part[warp] = (double)acc.hi + (double)acc.lo;
    if (clusters > 1 && attempt == 0) cluster_wait();
    __syncthreads();
    if ((int)threadIdx.x < clusters) {
      double sum = 0.0;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) sum += warp_part[w];
      if (clusters > 1)
        *cl.map_shared_rank(&cta_part[attempt][rank], threadIdx.x) = sum;
      else
        cta_part[attempt][0] = sum;
    }
    if (clusters > 1)
      cl.sync();
    else
      __syncthreads();
    // warp 0 finds the CTA and then the warp whose running sum passes the
    // mark, or the last that has any where rounding leaves none
    if (warp == 0) {
      const double part = lane < clusters ? cta_part[attempt][lane] : 0.0;
      double total = part;
#pragma unroll
      for (int o = kMaxCluster / 2; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      total = __shfl_sync(0xffffffffu, total, 0);
      const double mark = (double)u * total;
      double before = 0.0;
      int at = passes_at(part, clusters, mark, &before), w = -2;  // -2: another CTA draws
      const bool none = at < 0, end = at == clusters;
      if (end) at = last_positive(part, clusters);
      if (at == rank) {
        const double mine = lane < WARPS ? warp_part[lane] : 0.0;
        w = end ? WARPS : passes_at(mine, WARPS, mark, &before);
        if (w == WARPS) w = WARPS + last_positive(mine, WARPS);
      }
      if (lane == 0) {
        pick.warp = none ? -1 : w;
        pick.before = before;
        pick.mark = mark;
      }
    }
    __syncthreads();
    if (pick.warp == -1) {  // r is zero everywhere
      if (res.q != nullptr || res.sure >= 0) {
        // nothing of the target is left over the draft: draw from the target
        res.q = nullptr;
        res.sure = -1;
        continue;
      }
      if (rank == 0 && threadIdx.x == 0) out_tokens[row0 + a] = -1;
      return;
    }
    if (pick.warp < 0 || pick.warp % WARPS != warp) return;
    const bool rest = pick.warp >= WARPS;  // past the end: the last positive value of the warp
    double before = pick.before;
    const double mark = pick.mark;
    Pair round_sums[HELD];
    if constexpr (RV > 0) {
#pragma unroll
      for (int j = 0; j < RV; ++j) {
        round_sums[j] = Pair{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) add_exact(round_sums[j], r[j][i]);
        round_sums[j] = warp_sum_pair(round_sums[j]);
      }
    }
    int found = -1, positive = -1;
#pragma unroll
    for (int j = 0; j < (RV > 0 ? RV : rounds); ++j) {
      if constexpr (RV == 0) {
        r[0][0] = r[0][1] = r[0][2] = r[0][3] = 0.f;
        if (begin + 128ll * j < vocab) res.at4(begin + 128 * j, r[0]);
        round_sums[0] = Pair{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) add_exact(round_sums[0], r[0][i]);
        round_sums[0] = warp_sum_pair(round_sums[0]);
      }
      const Pair sum = round_sums[RV > 0 ? j : 0];
      if (!(sum.hi > 0.f) || found >= 0) continue;  // the same for all lanes
      const float* x = r[RV > 0 ? j : 0];
      const int v = begin + 128 * j;  // in the vocabulary wherever x is not zero
      const double round_sum = (double)sum.hi + (double)sum.lo;
      const bool here = !rest && before + round_sum > mark;
      if (!here) before += round_sum;
      int pos = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) pos = x[i] > 0.f ? v + i : pos;
      positive = __reduce_max_sync(0xffffffffu, pos);
      if (!here) continue;
      double inc[4];
      inc[0] = x[0];
#pragma unroll
      for (int i = 1; i < 4; ++i) inc[i] = inc[i - 1] + (double)x[i];
      double run = inc[3];  // inclusive sums over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
      }
      double lane_before = __shfl_up_sync(0xffffffffu, run, 1);
      if (lane == 0) lane_before = 0.0;
      lane_before += before;
      int hit = 0x7fffffff;
#pragma unroll
      for (int i = 3; i >= 0; --i) hit = x[i] > 0.f && lane_before + inc[i] > mark ? v + i : hit;
      hit = __reduce_min_sync(0xffffffffu, hit);
      found = hit == 0x7fffffff ? positive : hit;
    }
    if (lane == 0) out_tokens[row0 + a] = found >= 0 ? found : positive;
    return;
  }
}

// CTAs for one row of `vocab`, of at most `limit` elements each.
int cluster_for(long long rows, int vocab, int limit, int sms) {
  int c = 1;
  while (c < kMaxCluster && ((long long)c * limit < vocab || (rows * c * 2 <= 2 * sms && vocab / (2 * c) >= 2048)))
    c *= 2;
  return c;
}

template <typename... A>
cudaError_t launch_clustered(void (*kernel)(A...), long long rows, int cluster, int threads, cudaStream_t st,
                             A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * cluster));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool aligned_rows(const void* p, long long ld) { return !misaligned16(p) && ld % 4 == 0; }

}  // namespace

extern "C" ARMT_API armt_status armt_token_probs(const float* logits, int64_t ld_logits, const float* temperature,
                                                 int64_t n_rows, int32_t vocab, float* probs, int64_t ld_probs,
                                                 void* stream) {
  return guarded([&]() -> armt_status {
    if (vocab <= 0 || n_rows < 0) return refuse(ARMT_ERR_ARG, "sizes must be positive");
    if (n_rows > 0 && (logits == nullptr || probs == nullptr)) return refuse(ARMT_ERR_ARG, "NULL argument");
    if ((reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(probs) |
         reinterpret_cast<uintptr_t>(temperature)) & 3)
      return refuse(ARMT_ERR_ARG, "pointers must be 4-byte aligned");
    if (ld_logits < vocab || ld_probs < vocab) return refuse(ARMT_ERR_SHAPE, "a row distance must be at least vocab");
    if (logits == probs && ld_logits != ld_probs)
      return refuse(ARMT_ERR_SHAPE, "in place needs one row distance for both");
    if (n_rows > (1ll << 27) || vocab > (1 << 30) || ld_logits > (1ll << 40) || ld_probs > (1ll << 40))
      return refuse(ARMT_ERR_SHAPE, "sizes too large");
    int dev = 0, sms = 0;
    const armt_status s = ready_device(&dev, &sms);
    if (s != ARMT_OK) return s;
    if (n_rows == 0) return ARMT_OK;
    const bool vec = aligned_rows(logits, ld_logits) && aligned_rows(probs, ld_probs);
    constexpr int unit = 4 * kProbThreads;
    const int c = cluster_for(n_rows, vocab, 8 * unit, sms);
    int slice = (vocab + c - 1) / c;
    slice = (slice + 3) & ~3;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) {
      return launch_clustered(kernel, (long long)n_rows, c, kProbThreads, st, logits, (long long)ld_logits,
                              temperature, (int)vocab, slice, probs, (long long)ld_probs, c);
    };
    cudaError_t e;
    if (slice <= unit)
      e = vec ? go(token_probs_kernel<true, 1>) : go(token_probs_kernel<false, 1>);
    else if (slice <= 2 * unit)
      e = vec ? go(token_probs_kernel<true, 2>) : go(token_probs_kernel<false, 2>);
    else if (slice <= 4 * unit)
      e = vec ? go(token_probs_kernel<true, 4>) : go(token_probs_kernel<false, 4>);
    else if (slice <= 8 * unit)
      e = vec ? go(token_probs_kernel<true, 8>) : go(token_probs_kernel<false, 8>);
    else
      e = vec ? go(token_probs_kernel<true, 0>) : go(token_probs_kernel<false, 0>);
    return launch_status(e, "token probabilities");
  });
}

extern "C" ARMT_API armt_status armt_verify_drafts(const float* target, int64_t ld_target, const float* draft,
                                                   int64_t ld_draft, const int32_t* tokens, const int32_t* start,
                                                   const float* uniform, int32_t n_seqs, int64_t n_drafts,
                                                   int32_t vocab, int32_t* n_accepted, int32_t* out_tokens,
                                                   void* stream) {
  return guarded([&]() -> armt_status {
    if (vocab <= 0 || n_seqs < 0 || n_drafts < 0) return refuse(ARMT_ERR_ARG, "sizes must be positive");
    if (n_seqs > 0 && (target == nullptr || start == nullptr || uniform == nullptr || n_accepted == nullptr ||
                       out_tokens == nullptr || (tokens == nullptr && n_drafts > 0)))
      return refuse(ARMT_ERR_ARG, "NULL argument");
    if ((reinterpret_cast<uintptr_t>(target) | reinterpret_cast<uintptr_t>(draft) |
         reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(start) |
         reinterpret_cast<uintptr_t>(uniform) | reinterpret_cast<uintptr_t>(n_accepted) |
         reinterpret_cast<uintptr_t>(out_tokens)) & 3)
      return refuse(ARMT_ERR_ARG, "pointers must be 4-byte aligned");
    if (ld_target < vocab || (draft != nullptr && ld_draft < vocab))
      return refuse(ARMT_ERR_SHAPE, "a row distance must be at least vocab");
    if (n_seqs > (1 << 27) || n_drafts > (1ll << 30) || vocab > (1 << 30) || ld_target > (1ll << 31) ||
        (draft != nullptr && ld_draft > (1ll << 31)))
      return refuse(ARMT_ERR_SHAPE, "sizes too large");
    int dev = 0, sms = 0;
    const armt_status s = ready_device(&dev, &sms);
    if (s != ARMT_OK) return s;
    if (n_seqs == 0) return ARMT_OK;
    const bool vec = aligned_rows(target, ld_target) && (draft == nullptr || aligned_rows(draft, ld_draft));
    // 16 warps a CTA hold their parts while the batch leaves SMs free for it (1
    // x 4 drafts of 128,256: 11.3 us, 18.0 with 8 that do not); beyond that 8
    // warps that do not (64 x 6: 21 us, 35 with 16 that do).
    int c = cluster_for(n_seqs, vocab, 8 * 128 * 16, sms);
    const bool many = (long long)n_seqs * c > 2 * sms;
    const int round = 128 * (many ? 8 : 16);  // of all warps of a CTA
    const int rounds = (int)(((vocab + c - 1) / c + round - 1) / round);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    auto go = [&](auto kernel) {
      return launch_clustered(kernel, (long long)n_seqs, c, many ? 256 : 512, st, target, (long long)ld_target, draft,
                              (long long)ld_draft, tokens, start, uniform, (int)n_drafts, (int)vocab, rounds, vec,
                              n_accepted, out_tokens, c);
    };
    return launch_status(many          ? go(verify_drafts_kernel<8, 0>)
                         : rounds <= 2 ? go(verify_drafts_kernel<16, 2>)
                         : rounds <= 4 ? go(verify_drafts_kernel<16, 4>)
                         : rounds <= 8 ? go(verify_drafts_kernel<16, 8>)
                                       : go(verify_drafts_kernel<16, 0>),
                         "draft verification");
  });
}
