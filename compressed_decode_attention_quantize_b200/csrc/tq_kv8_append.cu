// Append to the 8-bit paged KV cache, with the position rotation on the way.
//
// For a new token at position p and coordinate pair (a, b) with the table
// entry (cos, sin) of p,  a' = a cos - b sin,  b' = a sin + b cos  (keys and
// queries; values are not rotated).  Per (page, kv head) and tensor:
//   s' = max(s, max |x| / 448)   over the page's new tokens (s = 0 when the
//                                token of slot 0 is among them),
//   code = e4m3(x / s'),   older codes of the page: e4m3(code * s / s').
// The statistics and the rotation are fp32; the one rounding is to e4m3.
//
// Bound by memory: every row is read once and every code written once.  A
// CTA takes one page of one sequence and a few of its 2 * Hkv (tensor, head)
// planes, about 1024 items of 16 coordinates, which stay in registers
// between the maximum and the coding; further CTAs rotate the query rows.
// There is one scale per page and plane and one CTA per page and plane, so no
// atomics reach device memory and the result has no order to depend on.
#include <algorithm>
#include <cfloat>

#include "tq_internal.h"
#include "tq_kv8.cuh"

namespace tqk {
namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_ITEMS = 4;                      // items per thread held in registers
constexpr int AP_ROUND = AP_THREADS * AP_ITEMS;  // items per round
constexpr int AP_QROWS = 32;                     // most query rows of a CTA

__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void load8(const __half* p, float* x) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float* x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Item c of a row: 16 coordinates in two runs of 8.  With the half-split
// rotation and c < rot / 16 the runs are (8c.., rot / 2 + 8c..), mates of one
// another; else they are neighbours.
__device__ __forceinline__ void item_runs(int c, int rot, int interleaved, int& e0, int& e1) {
  const bool mates = !interleaved && c < rot / 16;
  e0 = mates ? 8 * c : 16 * c;
  e1 = mates ? rot / 2 + 8 * c : 16 * c + 8;
}

// x[0..7], x[8..15]: the item's runs.  cs: the table row of the position.
__device__ __forceinline__ void rotate16(float* x, const float* cs, int c, int rot, int interleaved) {
  if (c >= rot / 16) return;
  float cv[8], sv[8];
  load8(cs + 8 * c, cv);
  load8(cs + rot / 2 + 8 * c, sv);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * cv[i] - b * sv[i];
      x[2 * i + 1] = a * sv[i] + b * cv[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[8 + i];
      x[i] = a * cv[i] - b * sv[i];
      x[8 + i] = a * sv[i] + b * cv[i];
    }
  }
}

// Eight codes of x / s.  s is 0 only where the whole page is: codes of 0.
__device__ __forceinline__ uint2 code8(const float* x, float s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = s > 0.f ? make_float2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s)) : make_float2(0.f, 0.f);
    w[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ uint32_t recode4(uint32_t w, float s_old, float s_new) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    const float2 g = make_float2(__fdiv_rn(f.x * s_old, s_new), __fdiv_rn(f.y * s_old, s_new));
    r |= (uint32_t)__nv_cvt_float2_to_fp8x2(g, __NV_SATFINITE, __NV_E4M3) << (16 * i);
  }
  return r;
}

// Rows [row0, row0 + count) of sequence b (clamped to [0, n]) and the position
// of the first of them.
__device__ __forceinline__ void seq_rows(const Kv8AppendArgs& a, int b, int64_t& row0, int& count, int64_t& start) {
  const int64_t r0 = min((int64_t)max(a.cu_q[b], 0), a.n), r1 = min((int64_t)max(a.cu_q[b + 1], 0), a.n);
  row0 = r0;
  count = (int)max((int64_t)0, r1 - r0);
  start = (int64_t)a.seq_lens[b] - count;
}

// Positions [lo, hi) of the sequence's rows that fall inside the cache.
__device__ __forceinline__ void seq_span(const Kv8AppendArgs& a, int count, int64_t start, int& lo, int& hi) {
  const int64_t cap = (int64_t)a.c.max_blocks * a.c.bs;
  const int64_t l = max(start, (int64_t)0), h = min(start + count, cap);
  lo = (int)min(l, cap);
  hi = (int)max(h, (int64_t)lo);
}

template <typename T>
__device__ void append_page(const Kv8AppendArgs& a, int64_t unit, int plane0, int nplanes) {
  __shared__ int s_warp[AP_THREADS / 32];
  __shared__ int s_b, s_j;
  __shared__ uint32_t s_amax[2 * 64];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = a.c.bs;
  // The unit-th touched page over all sequences.
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += AP_THREADS) {
    const int b = b0 + tid;
    int pages = 0, first = 0;
    if (b < a.B) {
      int64_t row0, start;
      int count, lo, hi;
      seq_rows(a, b, row0, count, start);
      seq_span(a, count, start, lo, hi);
      first = lo / bs;
      if (hi > lo) pages = (hi - 1) / bs - first + 1;
    }
    int incl = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    if (tid == 0) s_b = -1;
    __syncthreads();
    int64_t base = before, all = before;
#pragma unroll
    for (int w = 0; w < AP_THREADS / 32; ++w) {
      if (w < warp) base += s_warp[w];
      all += s_warp[w];
    }
    const int64_t at = base + incl - pages;
    if (unit >= at && unit < at + pages) {
      s_b = b;
      s_j = first + (int)(unit - at);
    }
    __syncthreads();
    if (s_b >= 0) break;
    before = all;
    if (b0 + AP_THREADS >= a.B) return;   // fewer pages than units
    __syncthreads();
  }
  const int b = s_b, j = s_j;
  const int32_t page = a.c.table[(int64_t)b * a.c.max_blocks + j];
  if (page < 0 || page >= a.c.num_blocks) return;
  int64_t row0, start;
  int count, lo, hi;
  seq_rows(a, b, row0, count, start);
  seq_span(a, count, start, lo, hi);
  const int p0 = max(lo, j * bs), p1 = min(hi, (j + 1) * bs);
  const int ntok = p1 - p0, slot0 = p0 - j * bs;
  row0 += p0 - start;
  const int per = a.d / 16;                // items per row
  const int64_t total = (int64_t)nplanes * ntok * per;
  if (tid < nplanes) s_amax[tid] = 0u;
  __syncthreads();

  auto load_item = [&](int64_t it, float* x, int& pl, int& tok, int& c) {
    c = (int)(it % per);
    const int r = (int)(it / per);
    tok = r % ntok;
    pl = r / ntok;
    const int plane = plane0 + pl;
    const bool key = plane < a.c.Hkv;
    const int h = key ? plane : plane - a.c.Hkv;
    const T* src = static_cast<const T*>(key ? a.k : a.v) + (row0 + tok) * (key ? a.ldk : a.ldv) + (int64_t)h * a.d;
    int e0, e1;
    item_runs(c, key ? a.rot : 0, a.interleaved, e0, e1);
    load8(src + e0, x);
    load8(src + e1, x + 8);
    if (key) rotate16(x, a.rope + (int64_t)(p0 + tok) * a.rot, c, a.rot, a.interleaved);
  };

  float x[AP_ITEMS][16];
  int pl[AP_ITEMS], tok[AP_ITEMS], cc[AP_ITEMS];
  const bool one_round = total <= AP_ROUND;
  for (int64_t r0 = 0; r0 < total; r0 += AP_ROUND) {
#pragma unroll
    for (int i = 0; i < AP_ITEMS; ++i) {
      const int64_t it = r0 + i * AP_THREADS + tid;
      if (it < total) {
        load_item(it, x[i], pl[i], tok[i], cc[i]);
        float m = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[i][e]));
        // Magnitudes order like their bit patterns.
        atomicMax(&s_amax[pl[i]], __float_as_uint(fminf(m, FLT_MAX)));
      }
    }
  }
  __syncthreads();
  // Older tokens of the page, where its scale grows.
  for (int p = 0; p < nplanes && slot0 > 0; ++p) {
    const int plane = plane0 + p;
    const bool key = plane < a.c.Hkv;
    const int h = key ? plane : plane - a.c.Hkv;
    const float s_old = (key ? a.c.kscale : a.c.vscale)[(int64_t)page * a.c.Hkv + h];
    const float s_new = fmaxf(s_old, __fdiv_rn(__uint_as_float(s_amax[p]), 448.f));
    if (s_new > s_old) {
      uint4* rows = reinterpret_cast<uint4*>((key ? a.c.kcodes : a.c.vcodes) +
                                             ((int64_t)page * a.c.Hkv + h) * bs * a.d);
      for (int i = tid; i < slot0 * per; i += AP_THREADS) {
        uint4 u = rows[i];
        u.x = recode4(u.x, s_old, s_new);
        u.y = recode4(u.y, s_old, s_new);
        u.z = recode4(u.z, s_old, s_new);
        u.w = recode4(u.w, s_old, s_new);
        rows[i] = u;
      }
    }
  }
  for (int64_t r0 = 0; r0 < total; r0 += AP_ROUND) {
#pragma unroll
    for (int i = 0; i < AP_ITEMS; ++i) {
      const int64_t it = r0 + i * AP_THREADS + tid;
      if (it < total) {
        if (!one_round) load_item(it, x[i], pl[i], tok[i], cc[i]);
        const int plane = plane0 + pl[i];
        const bool key = plane < a.c.Hkv;
        const int h = key ? plane : plane - a.c.Hkv;
        const int64_t ph = (int64_t)page * a.c.Hkv + h;
        float s = __fdiv_rn(__uint_as_float(s_amax[pl[i]]), 448.f);
        if (slot0 > 0) s = fmaxf(s, (key ? a.c.kscale : a.c.vscale)[ph]);
        int e0, e1;
        item_runs(cc[i], key ? a.rot : 0, a.interleaved, e0, e1);
        uint8_t* dst = (key ? a.c.kcodes : a.c.vcodes) + (ph * bs + slot0 + tok[i]) * a.d;
        *reinterpret_cast<uint2*>(dst + e0) = code8(x[i], s);
        *reinterpret_cast<uint2*>(dst + e1) = code8(x[i] + 8, s);
      }
    }
  }
  __syncthreads();   // every reader of the old scales is done
  if (tid < nplanes) {
    const int plane = plane0 + tid;
    const bool key = plane < a.c.Hkv;
    float* sc = (key ? a.c.kscale : a.c.vscale) + (int64_t)page * a.c.Hkv + (key ? plane : plane - a.c.Hkv);
    float s = __fdiv_rn(__uint_as_float(s_amax[tid]), 448.f);
    if (slot0 > 0) s = fmaxf(s, *sc);
    *sc = s;
  }
}

// Query rows [r0, r1): rotated by their position.  A row whose position is
// outside the cache becomes 0; rows of no sequence are left as they were.
template <typename T>
__device__ void rotate_queries(const Kv8AppendArgs& a, int64_t r0, int64_t r1) {
  __shared__ int s_pos[AP_QROWS];
  const int tid = threadIdx.x;
  if (tid < AP_QROWS) s_pos[tid] = -2;   // no sequence
  __syncthreads();
  const int64_t cap = (int64_t)a.c.max_blocks * a.c.bs;
  for (int b = tid; b < a.B; b += AP_THREADS) {
    int64_t row0, start;
    int count;
    seq_rows(a, b, row0, count, start);
    for (int64_t r = max(row0, r0); r < min(row0 + count, r1); ++r) {
      const int64_t p = start + (r - row0);
      s_pos[r - r0] = p >= 0 && p < cap ? (int)p : -1;
    }
  }
  __syncthreads();
  const int per = a.d / 16;
  const int64_t total = (r1 - r0) * a.Hq * per;
  for (int64_t it = tid; it < total; it += AP_THREADS) {
    const int c = (int)(it % per);
    const int64_t rh = it / per;
    const int h = (int)(rh % a.Hq);
    const int64_t r = rh / a.Hq;
    const int pos = s_pos[r];
    if (pos == -2) continue;
    const T* src = static_cast<const T*>(a.q) + (r0 + r) * a.ldq + (int64_t)h * a.d;
    T* dst = static_cast<T*>(a.q_out) + (r0 + r) * a.ldqo + (int64_t)h * a.d;
    int e0, e1;
    item_runs(c, a.rot, a.interleaved, e0, e1);
    float x[16];
    load8(src + e0, x);
    load8(src + e1, x + 8);
    if (pos >= 0) {
      rotate16(x, a.rope + (int64_t)pos * a.rot, c, a.rot, a.interleaved);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = 0.f;
    }
    store8(dst + e0, x);
    store8(dst + e1, x + 8);
  }
}

template <typename T>
__global__ void __launch_bounds__(AP_THREADS) k_kv8_append(Kv8AppendArgs a, int64_t kv_blocks, int planes, int qrows) {
  const int64_t blk = blockIdx.x;
  const int groups = (2 * a.c.Hkv + planes - 1) / planes;
  if (blk < kv_blocks) {
    const int g = (int)(blk % groups);
    append_page<T>(a, blk / groups, g * planes, min(planes, 2 * a.c.Hkv - g * planes));
  } else {
    const int64_t r0 = (blk - kv_blocks) * qrows;
    rotate_queries<T>(a, r0, min(a.n, r0 + qrows));
  }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t s) {
  // Touched pages: a sequence with c rows touches at most min(c, c / bs + 2).
  const int64_t units = std::min(a.n, a.n / a.c.bs + 2 * (int64_t)a.B);
  const int per = a.d / 16;
  // Rows of a page in this call: one per sequence and step, or whole pages.
  const int64_t rows = std::min((int64_t)a.c.bs, (a.n + a.B - 1) / a.B);
  int planes = (int)(AP_ROUND / (rows * per));
  planes = std::max(1, std::min({planes, 2 * a.c.Hkv, 128}));
  const int groups = (2 * a.c.Hkv + planes - 1) / planes;
  const int64_t kv_blocks = units * groups;
  int qrows = (int)std::max<int64_t>(1, std::min<int64_t>(AP_QROWS, 2 * AP_ROUND / ((int64_t)std::max(1, a.Hq) * per)));
  const int64_t blocks = kv_blocks + (a.q ? (a.n + qrows - 1) / qrows : 0);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (blocks == 0) return cudaSuccess;
  if (a.dtype == TQ_F32)
    k_kv8_append<float><<<(unsigned)blocks, AP_THREADS, 0, s>>>(a, kv_blocks, planes, qrows);
  else if (a.dtype == TQ_BF16)
    k_kv8_append<__nv_bfloat16><<<(unsigned)blocks, AP_THREADS, 0, s>>>(a, kv_blocks, planes, qrows);
  else
    k_kv8_append<__half><<<(unsigned)blocks, AP_THREADS, 0, s>>>(a, kv_blocks, planes, qrows);
  return cudaGetLastError();
}

}  // namespace tqk
