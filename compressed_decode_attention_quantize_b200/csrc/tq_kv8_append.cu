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
// planes, about 256 items of 16 coordinates, which stay in registers as they
// were read between the maximum and the coding (more of them are read twice;
// the rotation is done twice: held in fp32 they cost half of the CTAs that fit
// on an SM).  Further CTAs
// rotate the query rows; a thread takes the same coordinates of four heads, so
// that it reads the table once and has 128 bytes of rows in flight.
// There is one scale per page and plane and one CTA per page and plane, so no
// atomics reach device memory and the result has no order to depend on.
//
// Measured on a B200 (device time): 23317 rows of five prompts, 32 + 16 heads
// of 128, bf16: 119 us, 4.5 TB/s of the 6.46 that a copy reaches (more of the
// time waits for loads than issues: rows that do not fit a round are read and
// rotated twice); fp32 201 us, 5.0 TB/s; one row 5.2 us, 128 rows 6.0 us
// (latency: lengths, page, rows, maximum, codes, one after the other).
#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "tq_internal.h"
#include "tq_kv8.cuh"

namespace tqk {
namespace {

// Threads, items and blocks per SM: a block waits at its barriers for the
// lengths, the rows and the maximum, and other blocks fill the gaps.  23317 rows
// of five prompts (bf16 / fp16) and 7149 rows of d = 64 take
//   256 threads, 2 items, 3 blocks   131 / 142 us, 15.1 us
//   128 threads, 4 items, 6 blocks   131 / 129 us, 13.4 us
//   128 threads, 2 items, 5, 6, 7    133, 121, 119 / 133, 130, 129 us, 15.0, 16.1, 15.4 us
// (a page of 64 rows of 128 then takes two rounds and reads its rows twice, the
// second time from the L2 cache).
constexpr int AP_THREADS = 128;
constexpr int AP_ITEMS = 2;                      // items per thread held in registers
constexpr int AP_ROUND = AP_THREADS * AP_ITEMS;  // items per round
constexpr int AP_QROWS = 32;                     // most query rows of a CTA
constexpr int AP_HEADS = 4;                      // query heads of a thread

// Eight elements as they are in memory, and in fp32.
template <typename T>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
    if constexpr (sizeof(T) == 4) {
      const uint32_t v[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = __uint_as_float(w[i]);
        x[4 + i] = __uint_as_float(v[i]);
      }
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
};
__device__ __forceinline__ void load8(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
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

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// x[0..7], x[8..15]: the item's runs; cv, sv: its cosines and sines.
__device__ __forceinline__ void rotate16(float* x, const float* cv, const float* sv, int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * cv[i] - b * sv[i];
      x[2 * i + 1] = a * sv[i] + b * cv[i];
    }
  } else {
    // Two pairs an instruction.
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 a = make_float2(x[i], x[i + 1]), b = make_float2(x[8 + i], x[9 + i]);
      const float2 c = make_float2(cv[i], cv[i + 1]), s = make_float2(sv[i], sv[i + 1]);
      const float2 p = fma2(make_float2(-b.x, -b.y), s, mul2(a, c)), q = fma2(b, c, mul2(a, s));
      x[i] = p.x;
      x[i + 1] = p.y;
      x[8 + i] = q.x;
      x[9 + i] = q.y;
    }
  }
}

// A scale and what its quotients need.  x / s is the IEEE quotient: with r the
// rounded reciprocal, q = x r is corrected by its exact remainder, q - (q s -
// x) r (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990), which is the rounded quotient where s is far
// from the ends of the range and its fraction is not all ones; elsewhere the
// division is called.  (Divisions of all elements took a third of the time of
// a prompt.)
struct Scale {
  float s, r;   // r = 0: divide
};
__device__ __forceinline__ Scale make_scale(float s) {
  const uint32_t bits = __float_as_uint(s);
  const bool plain = s > 7.9e-31f && s < 1.2e30f && (bits & 0x7FFFFFu) != 0x7FFFFFu;
  Scale c;
  c.s = s;
  c.r = plain ? __frcp_rn(s) : 0.f;
  return c;
}
__device__ __forceinline__ float quotient(float x, const Scale& c) {
  const float q = x * c.r;
  return fmaf(fmaf(q, c.s, -x), -c.r, q);   // with these signs x = -0 gives -0
}

// Eight codes of x / s.  s is 0 only where the whole page is: codes of 0.
__device__ __forceinline__ uint2 code8(const float* x, const Scale& c) {
  uint32_t w[4];
  if (c.r != 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __nv_cvt_float2_to_fp8x2(make_float2(quotient(x[2 * i], c), quotient(x[2 * i + 1], c)), __NV_SATFINITE,
                                      __NV_E4M3);
  } else {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const float2 f = c.s > 0.f ? make_float2(__fdiv_rn(x[2 * i], c.s), __fdiv_rn(x[2 * i + 1], c.s)) : make_float2(0.f, 0.f);
      w[i] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
    }
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

template <typename T, int D>
__device__ void append_page(const Kv8AppendArgs& a, int64_t unit, int plane0, int nplanes) {
  __shared__ int s_warp[AP_THREADS / 32];
  __shared__ int s_b, s_j;
  __shared__ uint32_t s_amax[2 * 64];
  __shared__ Scale s_scale[2 * 64];
  __shared__ float s_before[2 * 64];
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
  constexpr uint32_t per = D / 16;                                       // items per row,
  const uint32_t perplane = ntok * per, total = nplanes * perplane;      // per plane, in all
  if (tid < nplanes) s_amax[tid] = 0u;
  __syncthreads();

  // Item `it`: its plane, token, run of coordinates and row in memory.
  struct Where {
    int pl, tok, c, e0, e1, h;
    bool key;
  };
  auto where = [&](uint32_t it) {
    Where w;
    w.pl = nplanes > 1 ? it / perplane : 0;
    const uint32_t r = it - w.pl * perplane;
    w.tok = r / per;
    w.c = r % per;
    w.key = plane0 + w.pl < a.c.Hkv;
    w.h = plane0 + w.pl - (w.key ? 0 : a.c.Hkv);
    item_runs(w.c, w.key ? a.rot : 0, a.interleaved, w.e0, w.e1);
    return w;
  };
  auto load = [&](const Where& w, Raw8<T>* u) {
    const T* src = static_cast<const T*>(w.key ? a.k : a.v) + (row0 + w.tok) * (w.key ? a.ldk : a.ldv) + w.h * D;
    u[0].load(src + w.e0);
    u[1].load(src + w.e1);
  };
  auto value = [&](const Where& w, const Raw8<T>* u, float* x) {
    u[0].get(x);
    u[1].get(x + 8);
    if (w.key && w.c < a.rot / 16) {
      const float* cs = a.rope + (int64_t)(p0 + w.tok) * a.rot + 8 * w.c;
      float cv[8], sv[8];
      load8(cs, cv);
      load8(cs + a.rot / 2, sv);
      rotate16(x, cv, sv, a.interleaved);
    }
  };

  // Largest magnitude of the item's plane; one atomic where the active lanes
  // share it.
  auto note = [&](int pl, uint32_t m) {
    const uint32_t act = __activemask();
    int same;
    __match_all_sync(act, pl, &same);
    if (same) {
      m = __reduce_max_sync(act, m);
      if (lane == __ffs(act) - 1) atomicMax(&s_amax[pl], m);
    } else {
      atomicMax(&s_amax[pl], m);
    }
  };

  Raw8<T> u[AP_ITEMS][2];
  const bool one_round = total <= AP_ROUND;
  for (uint32_t r0 = 0; r0 < total; r0 += AP_ROUND) {
#pragma unroll
    for (int i = 0; i < AP_ITEMS; ++i) {
      const uint32_t it = r0 + i * AP_THREADS + tid;
      if (it < total) load(where(it), u[i]);
    }
#pragma unroll
    for (int i = 0; i < AP_ITEMS; ++i) {
      const uint32_t it = r0 + i * AP_THREADS + tid;
      if (it < total) {
        const Where w = where(it);
        float x[16], m = 0.f;
        value(w, u[i], x);
#pragma unroll
        for (int e = 0; e < 16; ++e) m = fmaxf(m, fabsf(x[e]));
        // Magnitudes order like their bit patterns.
        note(w.pl, __float_as_uint(fminf(m, FLT_MAX)));
      }
    }
  }
  __syncthreads();
  // Old and new scales; the new ones are written here.
  if (tid < nplanes) {
    const int plane = plane0 + tid;
    const bool key = plane < a.c.Hkv;
    float* sc = (key ? a.c.kscale : a.c.vscale) + (int64_t)page * a.c.Hkv + (key ? plane : plane - a.c.Hkv);
    const float s_old = slot0 > 0 ? *sc : 0.f;
    const float s_new = fmaxf(s_old, __fdiv_rn(__uint_as_float(s_amax[tid]), 448.f));
    s_scale[tid] = make_scale(s_new);
    s_before[tid] = s_old;
    *sc = s_new;
  }
  __syncthreads();
  // Older tokens of the page, where its scale grows.
  for (int p = 0; p < nplanes && slot0 > 0; ++p) {
    const int plane = plane0 + p;
    const bool key = plane < a.c.Hkv;
    const int h = key ? plane : plane - a.c.Hkv;
    const float s_old = s_before[p], s_new = s_scale[p].s;
    if (s_new > s_old) {
      uint4* rows = reinterpret_cast<uint4*>((key ? a.c.kcodes : a.c.vcodes) +
                                             ((int64_t)page * a.c.Hkv + h) * bs * D);
      for (int i = tid; i < slot0 * (int)per; i += AP_THREADS) {
        uint4 v = rows[i];
        v.x = recode4(v.x, s_old, s_new);
        v.y = recode4(v.y, s_old, s_new);
        v.z = recode4(v.z, s_old, s_new);
        v.w = recode4(v.w, s_old, s_new);
        rows[i] = v;
      }
    }
  }
  for (uint32_t r0 = 0; r0 < total; r0 += AP_ROUND) {
#pragma unroll
    for (int i = 0; i < AP_ITEMS; ++i) {
      const uint32_t it = r0 + i * AP_THREADS + tid;
      if (it < total) {
        const Where w = where(it);
        if (!one_round) load(w, u[i]);
        float x[16];
        value(w, u[i], x);
        const int64_t ph = (int64_t)page * a.c.Hkv + w.h;
        const Scale s = s_scale[w.pl];
        uint8_t* dst = (w.key ? a.c.kcodes : a.c.vcodes) + (ph * bs + slot0 + w.tok) * D;
        *reinterpret_cast<uint2*>(dst + w.e0) = code8(x, s);
        *reinterpret_cast<uint2*>(dst + w.e1) = code8(x + 8, s);
      }
    }
  }
}

// Query rows [r0, r1): rotated by their position.  A row whose position is
// outside the cache becomes 0; rows of no sequence are left as they were.
template <typename T, int D>
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
  // A thread takes one run of coordinates of AP_HEADS heads of a row.
  constexpr uint32_t per = D / 16;
  const uint32_t groups = (a.Hq + AP_HEADS - 1) / AP_HEADS, total = (uint32_t)(r1 - r0) * groups * per;
  for (uint32_t it = tid; it < total; it += AP_THREADS) {
    const uint32_t rg = it / per, c = it % per, r = rg / groups, h0 = (rg - r * groups) * AP_HEADS;
    const int pos = s_pos[r];
    if (pos == -2) continue;
    int e0, e1;
    item_runs(c, a.rot, a.interleaved, e0, e1);
    const T* src = static_cast<const T*>(a.q) + (r0 + r) * a.ldq + h0 * D;
    T* dst = static_cast<T*>(a.q_out) + (r0 + r) * a.ldqo + h0 * D;
    const int heads = min(AP_HEADS, a.Hq - (int)h0);
    Raw8<T> u[AP_HEADS][2];
#pragma unroll
    for (int k = 0; k < AP_HEADS; ++k)
      if (k < heads) {
        u[k][0].load(src + k * D + e0);
        u[k][1].load(src + k * D + e1);
      }
    float cv[8], sv[8];
    const bool turn = pos >= 0 && (int)c < a.rot / 16;
    if (turn) {
      const float* cs = a.rope + (int64_t)pos * a.rot + 8 * c;
      load8(cs, cv);
      load8(cs + a.rot / 2, sv);
    }
#pragma unroll
    for (int k = 0; k < AP_HEADS; ++k)
      if (k < heads) {
        float x[16];
        u[k][0].get(x);
        u[k][1].get(x + 8);
        if (turn) rotate16(x, cv, sv, a.interleaved);
        if (pos < 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0.f;
        }
        store8(dst + k * D + e0, x);
        store8(dst + k * D + e1, x + 8);
      }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(AP_THREADS, sizeof(T) == 4 ? 4 : 7) k_kv8_append(Kv8AppendArgs a, int64_t kv_blocks, int planes, int qrows) {
  const int64_t blk = blockIdx.x;
  const int groups = (2 * a.c.Hkv + planes - 1) / planes;
  if (blk < kv_blocks) {
    const int g = (int)(blk % groups);
    append_page<T, D>(a, blk / groups, g * planes, min(planes, 2 * a.c.Hkv - g * planes));
  } else {
    const int64_t r0 = (blk - kv_blocks) * qrows;
    rotate_queries<T, D>(a, r0, min(a.n, r0 + qrows));
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
  // Two turns of a CTA's threads.
  const int qitems = std::max(1, (a.Hq + AP_HEADS - 1) / AP_HEADS * per);
  const int qrows = std::max(1, std::min(AP_QROWS, 2 * AP_THREADS / qitems));
  const int64_t blocks = kv_blocks + (a.q ? (a.n + qrows - 1) / qrows : 0);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (blocks == 0) return cudaSuccess;
  auto run = [&](auto* kernel) { kernel<<<(unsigned)blocks, AP_THREADS, 0, s>>>(a, kv_blocks, planes, qrows); };
  if (a.dtype == TQ_F32)
    a.d == 128 ? run(k_kv8_append<float, 128>) : run(k_kv8_append<float, 64>);
  else if (a.dtype == TQ_BF16)
    a.d == 128 ? run(k_kv8_append<__nv_bfloat16, 128>) : run(k_kv8_append<__nv_bfloat16, 64>);
  else
    a.d == 128 ? run(k_kv8_append<__half, 128>) : run(k_kv8_append<__half, 64>);
  return cudaGetLastError();
}

}  // namespace tqk
