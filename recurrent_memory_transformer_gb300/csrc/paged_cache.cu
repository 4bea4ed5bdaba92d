// Writing new rows into the paged cache and reading them back.
//
// Both are copies: 2 n Hkv (2 hd + stored bytes) bytes and nothing else to
// do, so HBM bounds them, and launch and load latency when n is a few rows.
// One warp moves one row of all kv heads, keys and values: a lane owns 8
// elements of a head (16 bytes of bf16, 8 codes), so a head's row is 8 or 16
// lanes, its largest magnitude takes 3 or 4 shuffles, and a warp has up to
// 8 16-byte loads in flight before the first store.  The sequence of a row is
// found by a 33-ary search of row_start over the warp's lanes (one or two
// dependent loads up to 1,024 sequences) while the row itself is on its way.
#include "paged.cuh"

using namespace armt;

namespace {

// The sequence that row r belongs to where starts are in order: the last b with
// row_start[b] <= r (otherwise some b in range; the caller checks that r lies in
// it, and looks at all if not).
__device__ __forceinline__ int find_seq(const int32_t* row_start, int n_seqs, int r, int lane) {
  int lo = 0, hi = n_seqs;  // row_start[lo] <= r is taken for granted; the answer is in [lo, hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 32) / 33;  // lanes look at lo + step, lo + 2 step, ...
    const int at = lo + (lane + 1) * step;
    const bool le = at < hi && row_start[at] <= r;
    const int k = __popc(__ballot_sync(0xffffffffu, le));
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

// The first sequence that has row r among the rows that a call treats, -1 if
// none has.  For rows the search finds no sequence for: padding, rows past max_new,
// and starts out of order.  128 sequences a round, whose loads are on their way
// together (1,000 sequences and 24 rows of padding: 11 us, 19 with 32, 9 without).
__device__ __noinline__ int scan_seqs(const int32_t* row_start, int n_seqs, int n_rows, int max_new, int r, int lane) {
  for (int b0 = 0; b0 < n_seqs; b0 += 128) {
    int first[4], end[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = b0 + 32 * j + lane;
      first[j] = b < n_seqs ? row_start[b] : -1;
      end[j] = b < n_seqs ? row_start[b + 1] : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool has = first[j] >= 0 && first[j] <= r && r < end[j] && end[j] <= n_rows && r - first[j] < max_new;
      const uint32_t which = __ballot_sync(0xffffffffu, has);
      if (which != 0) return b0 + 32 * j + __ffs((int)which) - 1;
    }
  }
  return -1;
}

// The largest |x| of a head's row, as bf16 bits (which order like the values;
// 0x7f80 and up: something is not finite), for its HD / 8 lanes.
template <int HD>
__device__ __forceinline__ uint32_t head_top(const uint4& x) {
  uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int o = HD / 16; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
// Largest finite |x| over a head's lanes, where some are not finite.
template <int HD>
__device__ __forceinline__ float head_max(float m) {
#pragma unroll
  for (int o = HD / 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Least E >= -100 with m <= 448 * 2^E = 0.875 * 2^(E + 9), for finite m >= 0.
// m = f * 2^x with 1 <= f < 2: 448 * 2^E >= m means E = x - 8, or x - 7 when
// f > 1.75 (a subnormal m has x = -127 here and takes -100 anyway).
__device__ __forceinline__ int scale_exp(float m) {
  const uint32_t u = __float_as_uint(m);
  const int x = (int)(u >> 23) - 127;
  return max(-100, x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0));
}

// 8 bf16 -> 8 codes of x * inv (inv = 2^-e).
__device__ __forceinline__ uint2 quantise8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = __fmul2_rn(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u)),
                                make_float2(inv, inv));
    c[i] = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// The same with the NaN code for what is not finite (saturation would turn
// infinity into 448).
__device__ __noinline__ uint2 quantise8_odd(uint4 x, float inv) {
  const uint2 q = quantise8(x, inv);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if ((w[i >> 1] >> (16 * (i & 1)) & 0x7f80u) == 0x7f80u)
      c[i >> 2] = (c[i >> 2] & ~(0xffu << (8 * (i & 3)))) | (0x7fu << (8 * (i & 3)));
  return make_uint2(c[0], c[1]);
}

__device__ __forceinline__ float finite_max8(const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = (w[i] << 16) & 0x7fffffffu, hi = w[i] & 0x7fff0000u;
    if (lo < 0x7f800000u) m = fmaxf(m, __uint_as_float(lo));
    if (hi < 0x7f800000u) m = fmaxf(m, __uint_as_float(hi));
  }
  return m;
}

// 8 codes -> 8 bf16 of code * scale (exact: a code has 4 significant bits and
// the product stays above bf16's smallest normal number).
__device__ __forceinline__ uint4 expand8(const uint2& c, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t word = i < 2 ? c.x : c.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(word >> (16 * (i & 1))), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    o[i] = pack_bf16x2(f.x * scale, f.y * scale);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

constexpr int kWarps = 4;
constexpr int kPieces = 4;  // 16-byte pieces of k (and of v) a lane holds at once

// Position of row r, and its page (-1: none; out of the batch: b = -1).
struct Place {
  int b, page, slot;
};
__device__ __forceinline__ Place place_of(const PagedView& p, int r, int lane) {
  Place t;
  t.b = find_seq(p.row_start, p.n_seqs, r, lane);
  PagedSeq s = paged_seq(p, t.b);
  int i = r - s.row0;
  if (i < 0 || i >= s.n || i >= p.max_new) {
    t.b = scan_seqs(p.row_start, p.n_seqs, p.n_rows, p.max_new, r, lane);
    if (t.b < 0) {
      t.page = t.slot = -1;
      return t;
    }
    s = paged_seq(p, t.b);
    i = r - s.row0;
  }
  const long long pos = (long long)s.kv_len - s.n + i;
  t.page = paged_page(p, t.b, pos);
  t.slot = (int)(pos & ((1 << p.page_shift) - 1));
  return t;
}

template <int HD, int TYPE>
__global__ void __launch_bounds__(kWarps * 32) cache_write_kernel(const bf16* __restrict__ k, long long k_stride,
                                                                  const bf16* __restrict__ v, long long v_stride,
                                                                  const PagedView p) {
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= p.n_rows) return;
  const int pieces = p.hkv * (HD / 8);  // per pool
  const uint4* ks = reinterpret_cast<const uint4*>(k + (long long)r * k_stride);
  const uint4* vs = reinterpret_cast<const uint4*>(v + (long long)r * v_stride);
  Place t;
  t.b = -2;
  for (int c0 = 0; c0 < pieces; c0 += 32 * kPieces) {
    uint4 kx[kPieces], vx[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int c = c0 + 32 * j + lane;
      kx[j] = vx[j] = make_uint4(0, 0, 0, 0);
      if (c < pieces) {
        kx[j] = __ldg(ks + c);
        vx[j] = __ldg(vs + c);
      }
    }
    if (t.b == -2) t = place_of(p, r, lane);  // the same for the whole warp
    if (t.page < 0) return;
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int c = c0 + 32 * j + lane;
      if (c0 + 32 * j >= pieces) break;  // warp-uniform: the shuffles below have all lanes
      const int head = c / (HD / 8), part = c % (HD / 8);
      const long long row = paged_row(p, t.page, head, t.slot);
      if constexpr (TYPE == ARMT_CACHE_BF16) {
        if (c < pieces) {
          reinterpret_cast<uint4*>(p.k)[row * (HD / 8) + part] = kx[j];
          reinterpret_cast<uint4*>(p.v)[row * (HD / 8) + part] = vx[j];
        }
      } else {
        const uint32_t kt = head_top<HD>(kx[j]), vt = head_top<HD>(vx[j]);
        // a row with something that is not finite takes the longer way, its whole warp with it
        const bool odd = __any_sync(0xffffffffu, max(kt, vt) >= 0x7f80u);
        float km = __uint_as_float(kt << 16), vm = __uint_as_float(vt << 16);
        if (odd) {
          km = head_max<HD>(finite_max8(kx[j]));
          vm = head_max<HD>(finite_max8(vx[j]));
        }
        const int ke = scale_exp(km), ve = scale_exp(vm);
        if (c < pieces) {
          const float ki = scale_of(127 - ke), vi = scale_of(127 - ve);
          reinterpret_cast<uint2*>(p.k)[row * (HD / 8) + part] = odd ? quantise8_odd(kx[j], ki) : quantise8(kx[j], ki);
          reinterpret_cast<uint2*>(p.v)[row * (HD / 8) + part] = odd ? quantise8_odd(vx[j], vi) : quantise8(vx[j], vi);
          if (part == 0) {
            p.k_scale[row] = (uint8_t)(ke + 127);
            p.v_scale[row] = (uint8_t)(ve + 127);
          }
        }
      }
    }
  }
}

template <int HD, int TYPE>
__global__ void __launch_bounds__(kWarps * 32) cache_read_kernel(bf16* __restrict__ k, long long k_stride,
                                                                 bf16* __restrict__ v, long long v_stride,
                                                                 const PagedView p) {
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= p.n_rows) return;
  const int pieces = p.hkv * (HD / 8);
  uint4* kd = reinterpret_cast<uint4*>(k + (long long)r * k_stride);
  uint4* vd = reinterpret_cast<uint4*>(v + (long long)r * v_stride);
  const Place t = place_of(p, r, lane);
  if (t.b < 0) return;
  for (int c0 = 0; c0 < pieces; c0 += 32 * kPieces) {
    uint4 kx[kPieces], vx[kPieces];
    uint32_t kb[kPieces], vb[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int c = c0 + 32 * j + lane;
      kx[j] = vx[j] = make_uint4(0, 0, 0, 0);
      kb[j] = vb[j] = 0;
      if (c < pieces && t.page >= 0) {
        const long long row = paged_row(p, t.page, c / (HD / 8), t.slot);
        const long long at = row * (HD / 8) + c % (HD / 8);
        if constexpr (TYPE == ARMT_CACHE_BF16) {
          kx[j] = reinterpret_cast<const uint4*>(p.k)[at];
          vx[j] = reinterpret_cast<const uint4*>(p.v)[at];
        } else {
          const uint2 a = reinterpret_cast<const uint2*>(p.k)[at], b = reinterpret_cast<const uint2*>(p.v)[at];
          kx[j].x = a.x, kx[j].y = a.y, vx[j].x = b.x, vx[j].y = b.y;
          kb[j] = p.k_scale[row];
          vb[j] = p.v_scale[row];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int c = c0 + 32 * j + lane;
      if (c >= pieces) break;
      if constexpr (TYPE == ARMT_CACHE_BF16) {
        kd[c] = kx[j];
        vd[c] = vx[j];
      } else {
        kd[c] = expand8(make_uint2(kx[j].x, kx[j].y), scale_of(kb[j]));
        vd[c] = expand8(make_uint2(vx[j].x, vx[j].y), scale_of(vb[j]));
      }
    }
  }
}

// Runs f(head_dim, type) with both as compile-time constants.
template <typename F>
void by_shape(const armt_kv_cache& c, F f) {
  using std::integral_constant;
  if (c.type == ARMT_CACHE_BF16)
    c.head_dim == 64 ? f(integral_constant<int, 64>(), integral_constant<int, ARMT_CACHE_BF16>())
                     : f(integral_constant<int, 128>(), integral_constant<int, ARMT_CACHE_BF16>());
  else
    c.head_dim == 64 ? f(integral_constant<int, 64>(), integral_constant<int, ARMT_CACHE_E4M3>())
                     : f(integral_constant<int, 128>(), integral_constant<int, ARMT_CACHE_E4M3>());
}

}  // namespace

extern "C" ARMT_API armt_status armt_cache_write_bf16(const void* k, int64_t k_stride, const void* v,
                                                      int64_t v_stride, const armt_kv_cache* cache,
                                                      const armt_paged_batch* batch, void* stream) {
  return guarded([&]() -> armt_status {
    armt_status s;
    if ((s = check_cache(cache)) != ARMT_OK || (s = check_batch(batch, cache)) != ARMT_OK) return s;
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    if ((s = check_rows(k, batch->n_rows, k_stride, width, "k")) != ARMT_OK || (s = check_rows(v, batch->n_rows, v_stride, width, "v")) != ARMT_OK)
      return s;
    int dev = 0, sms = 0;
    if ((s = ready_device(&dev, &sms)) != ARMT_OK) return s;
    if (batch->n_rows == 0) return ARMT_OK;
    const PagedView view = paged_view(*cache, *batch);
    const unsigned grid = (unsigned)((batch->n_rows + kWarps - 1) / kWarps);
    by_shape(*cache, [&](auto hd, auto type) {
      cache_write_kernel<hd(), type()><<<grid, kWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
          static_cast<const bf16*>(k), k_stride, static_cast<const bf16*>(v), v_stride, view);
    });
    return launch_status(cudaGetLastError(), "cache write");
  });
}

extern "C" ARMT_API armt_status armt_cache_read_bf16(const armt_kv_cache* cache, const armt_paged_batch* batch,
                                                     void* k, int64_t k_stride, void* v, int64_t v_stride,
                                                     void* stream) {
  return guarded([&]() -> armt_status {
    armt_status s;
    if ((s = check_cache(cache)) != ARMT_OK || (s = check_batch(batch, cache)) != ARMT_OK) return s;
    const int64_t width = (int64_t)cache->n_kv_heads * cache->head_dim;
    if ((s = check_rows(k, batch->n_rows, k_stride, width, "k")) != ARMT_OK || (s = check_rows(v, batch->n_rows, v_stride, width, "v")) != ARMT_OK)
      return s;
    int dev = 0, sms = 0;
    if ((s = ready_device(&dev, &sms)) != ARMT_OK) return s;
    if (batch->n_rows == 0) return ARMT_OK;
    const PagedView view = paged_view(*cache, *batch);
    const unsigned grid = (unsigned)((batch->n_rows + kWarps - 1) / kWarps);
    by_shape(*cache, [&](auto hd, auto type) {
      cache_read_kernel<hd(), type()><<<grid, kWarps * 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
          static_cast<bf16*>(k), k_stride, static_cast<bf16*>(v), v_stride, view);
    });
    return launch_status(cudaGetLastError(), "cache read");
  });
}
