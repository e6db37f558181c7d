// Decode attention over the 8-bit paged KV cache: one query row per sequence,
// or a few (drafted tokens).
//
// For query head h of sequence b, kv head g, key code k_t with page scale a_t
// and value code v_t with page scale w_t:
//   x_t = scale log2(e) a_t <q, k_t>,   out = sum_t 2^x_t w_t v_t / sum_t 2^x_t
// over the valid tokens t.  With M a reference near the maximum of x_t +
// log2(w_t),
//   O = sum_t 2^(x_t + log2 w_t - M) v_t,   L = sum_t 2^(x_t + log2 w_t - M) / w_t
// and out = O / L.  M is 2^8 below the maximum of the first tile and stays until
// a weight passes 2^14: so the weights fit binary16 whatever the pages' scales
// are, a tile takes no maximum and no exchange between lanes, and the value
// codes enter the product exactly.  The one rounding is that of the weights to
// binary16 (relative 2^-11; below 2^-14 half a step of 2^-24, which is 2^-33 of
// the largest weight or less).  The queries
// are scaled by a power of two per row so that binary16 holds them exactly as
// well (bf16 rows down to 2^-32 of their largest element); products accumulate
// in fp32.
//
// Bound by memory: 2 d bytes per token and kv head.  A warp is the unit of
// work.  The tiles (16 tokens, or 32) of all (sequence, block, kv head) form one
// list that the warps of a persistent grid share in equal contiguous ranges, so
// ragged batches and single long sequences balance alike.  Each warp runs its
// own ring of tiles, filled by TMA (swizzled rows; the same pieces copied with
// cp.async stopped at 4.5 TB/s, whatever the warps and stages).  The d axes of
// both products and the order of the tokens are permuted so that every lane
// reads its operands in pieces of 16 bytes (8 for values of d = 64) without
// bank conflicts.  Both products are taken transposed, S^T = K Q^T and O^T =
// V^T P^T: the 16 rows of a matrix instruction are then tokens and coordinates
// and its 8 columns are query heads (times query rows, where a sequence has
// several: a block of columns is as many whole rows as fit), so a group of up
// to 8 heads leaves no part of it empty.  (mma.sync, not tcgen05: 8 or 16
// columns would fill 1/16 of a 128-row tile, and the tensor pipes are 10 to
// 20% busy.)  A warp that holds a whole pair writes the output; the parts of
// the others are joined in the CTA's shared memory, and only what crosses CTAs
// is left as (O, M, L) for k_kv8_merge.
//
// Measured on a B200 (device time): 16 x 32768 tokens, 8 kv heads, d = 128:
// 188 to 195 us over runs, 5.5 to 5.7 TB/s of the 6.46 that a copy reaches; 4 x
// 131072: 184 to 192 us.  67 ragged sequences, d = 64: 53 to 54 us (3.0 TB/s:
// bound by the instructions of a tile); 16 x 4 rows of 4 heads over up to 8104
// tokens, d = 128: 63 to 64 us.  12, 16 and 20 warps and 2 to 4 stages are within
// 4% of one another; 32 tokens at a time in the products spill at d = 128.
#include <cuda.h>

#include <algorithm>

#include "tq_internal.h"
#include "tq_kv8.cuh"
#include "tq_tc_common.cuh"

namespace tqk {

__device__ int g_kv8_decode_fault = 0;

namespace {

constexpr int DEC_WARPS = 12;
constexpr int DEC_STAGES = 4;
constexpr int MERGE_THREADS = 256;        // and the most CTAs of a decode
// M is set this far below a maximum (log2), so the largest weight is at least
// 2^8: binary16 then takes weights down to 2^-33 of it, of which a long tail may
// be made, and the fp32 sums do not mind.  (Ragged sequences 53.9 us, with M at
// the maximum 53.5 us.)
constexpr float kBelow = 8.f;

__device__ __forceinline__ uint32_t s_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// The tokens (a box of the map) whose first row is `row` to shared memory.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(addr) : "memory");
  return u;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 u;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(u.x), "=r"(u.y) : "r"(addr) : "memory");
  return u;
}

// Two e4m3 codes (low and high byte of a half word) to binary16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2hi_to_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}\n" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight elements from i (a multiple of 8), zeros if not `in`.
__device__ __forceinline__ void load_q8(const void* q, int dtype, int64_t i, bool in, float* x) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (in) u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(q) + i));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (dtype == TQ_BF16) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      x[2 * k] = f.x;
      x[2 * k + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t i, float a, float b) {
  if (dtype == TQ_BF16)
    *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(out) + i) = __floats2bfloat162_rn(a, b);
  else
    *reinterpret_cast<__half2*>(static_cast<__half*>(out) + i) = __floats2half2_rn(a, b);
}

// One ring stage of a warp, a tile: 16 S rows of D key codes, then 16 S of value codes.
template <int D, int S>
__host__ __device__ constexpr int stage_bytes() { return 32 * D * S; }
// Piece `c` of 16 bytes of token r, as TMA's swizzle of 128-byte rows places
// it; with d = 64 a row holds two tokens.
template <int D>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  const int row = D == 128 ? r : r >> 1, unit = D == 128 ? c : 4 * (r & 1) + c;
  return row * 128 + ((unit ^ (row & 7)) << 4);
}
// Token of row k (0..7) of a matrix operand: chosen so that the lanes of one
// access differ in the bits that the swizzle turns into other banks.
template <int D>
__device__ __forceinline__ int token_of(int k) {
  return D == 128 ? k ^ ((k & 1) << 2) : k ^ ((k >> 1) & 1);
}

// Turn of a record's pieces: lanes with different columns then store to
// different banks.
template <int D>
__device__ __forceinline__ int record_turn(int c) {
  return D == 128 ? (c >> 1) & 3 : ((c >> 1) & 1) | (((c >> 2) & 1) << 2);
}

// Shared memory of the decode kernel.
template <int D, int S>
struct DecLayout {
  static constexpr int scales = DEC_WARPS * DEC_STAGES * stage_bytes<D, S>();   // float2 [warp][stage]
  static constexpr int bars = scales + DEC_WARPS * DEC_STAGES * 8;
  static constexpr int prefix = bars + DEC_WARPS * DEC_STAGES * 8;           // int64 [B + 1]
  static constexpr int total(int B) { return prefix + (B + 1) * 8 + 1024; }  // + alignment slack
};

// A block of columns: the query rows [row0, row0 + ntok) of a sequence, column
// c being row c / G and head c % G of the kv group.
struct Block {
  int row0, ntok, pos0;     // position of the first row
  int lo, hi;               // tokens that any row sees
  int all_lo, all_hi;       // tokens that every row sees
  __device__ int tiles(int T) const { return hi > lo ? (hi + T - 1) / T - lo / T : 0; }   // of T tokens
};
__device__ __forceinline__ void seq_of(const Kv8AttnArgs& a, int b, int& row0, int& count, int& start) {
  if (a.cu_q) {
    ragged_seq(a, b, row0, count, start);
  } else {
    row0 = b;
    count = 1;
    start = first_pos(a, b, 1);
  }
}
__device__ __forceinline__ Block block_of(const Kv8AttnArgs& a, int row0, int count, int start, int k, int per) {
  Block v;
  const int cap = a.c.max_blocks * a.c.bs;
  v.row0 = row0 + k * per;
  v.ntok = min(count - k * per, per);
  v.pos0 = start + k * per;
  const int last = v.pos0 + v.ntok - 1;
  v.hi = min(max(last + 1, 0), cap);
  v.lo = a.window > 0 ? min(max(v.pos0 - a.window + 1, 0), v.hi) : 0;
  v.all_hi = min(max(v.pos0 + 1, 0), cap);
  v.all_lo = a.window > 0 ? max(last - a.window + 1, 0) : 0;
  return v;
}

// One warp's attention of the columns of one block and kv head over a run of
// tokens.  Columns of the matrix products come in R groups of 8.  Lane (g =
// lane / 4, qd = lane % 4) holds the scores of rows g, g + 8 (tokens
// token_of(g), + 8) and columns 2 qd, 2 qd + 1 of each group.
template <int D, int R, int S>
struct Attend {
  static constexpr int NJ = D / 16;         // matrix instructions over d
  uint32_t qb[NJ][R][2];                    // query operands: column g of each group
  float qf[R][2];                           // scale log2(e) / the column's power of two
  float o[NJ][R][4];                        // (d even, odd) x (column 2 qd, 2 qd + 1) as [2 * odd + column]
  float m[R][2], l[R][2];
  int clo[R][2], chi[R][2];                 // tokens that the column sees
  uint32_t koff[2], voff[4];                // the lane's pieces of a stage
  bool begun;

  __device__ void place(int lane) {
    const int g = lane >> 2, qd = lane & 3;
#pragma unroll
    for (int r = 0; r < 2; ++r) koff[r] = piece_at<D>(token_of<D>(g) + 8 * r, qd);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = token_of<D>(2 * qd + (r & 1)) + 8 * (r >> 1);
      voff[r] = 16 * S * D + (D == 128 ? piece_at<D>(tok, g) : piece_at<D>(tok, g >> 1) + 8 * (g & 1));
    }
  }

  // Offset of a column's row in q and out.
  __device__ static int64_t column(const Kv8AttnArgs& a, const Block& v, int h, int c) {
    const int tok = c / a.G;
    return ((int64_t)(v.row0 + tok) * a.Hq + (int64_t)h * a.G + (c - tok * a.G)) * D;
  }

  __device__ void load_queries(const Kv8AttnArgs& a, const Block& v, int h, int lane) {
    const int g = lane >> 2, qd = lane & 3, ncols = v.ntok * a.G;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int col = g + 8 * r;
      const int64_t base = column(a, v, h, col);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 8 * r + 2 * qd + i, p = v.pos0 + c / a.G;
        // A column of nothing sees all that the block sees: its sums stay finite.
        clo[r][i] = c < ncols && a.window > 0 ? max(p - a.window + 1, 0) : v.lo;
        chi[r][i] = c < ncols ? min(p + 1, v.hi) : v.hi;
      }
      float x[D / 4];
      float mx = 0.f;
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int i = 0; i < 16; i += 8) {
          load_q8(a.q, a.dtype, base + 64 * c + 16 * qd + i, col < ncols, x + 16 * c + i);
#pragma unroll
          for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(x[16 * c + i + k]));
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      // 2^e with mx 2^e in [2^14, 2^15), in two factors that fp32 can hold.
      const int e = mx > 0.f ? 14 - (min(max((int)((__float_as_uint(mx) >> 23) & 255), 1), 254) - 127) : 0;
      const int e1 = e / 2, e2 = e - e1;
      const float f1 = __uint_as_float((uint32_t)(127 + e1) << 23), f2 = __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
      for (int s = 0; s < NJ; ++s)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = 16 * (s / 4) + 4 * (s % 4) + 2 * k;
          const __half2 w = __floats2half2_rn(x[i] * f1 * f2, x[i + 1] * f1 * f2);
          qb[s][r][k] = *reinterpret_cast<const uint32_t*>(&w);
        }
      const float f = a.scale_log2 / f1 / f2;
      qf[r][0] = __shfl_sync(0xffffffffu, f, 8 * qd);
      qf[r][1] = __shfl_sync(0xffffffffu, f, 8 * qd + 4);
    }
  }

  __device__ void reset() {
    begun = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[r][i] = -INFINITY;
        l[r][i] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[j][r][i] = 0.f;
    }
  }

  // Copy the 16 S tokens from `slot` of page `page` (or nothing, if it is not a
  // page) into a stage, and the page's scales (-1 where there is no page).
  __device__ static void issue(const Kv8AttnArgs& a, const CUtensorMap* mk, const CUtensorMap* mv, uint32_t st,
                               uint32_t scales, uint32_t bar, int32_t page, int h, int slot, int lane) {
    const bool ok = page >= 0 && page < a.c.num_blocks;
    const int ph = ok ? page * a.c.Hkv + h : 0;   // rows stay below 2^31
    if (ok) {
      const int row = (ph * a.c.bs + slot) / (128 / D);
      if (elect_one()) {
        mbar_expect_tx(bar, stage_bytes<D, S>());
        tma_rows(st, mk, row, bar);
        tma_rows(st + 16 * S * D, mv, row, bar);
      }
    } else if (elect_one()) {
      mbar_arrive(bar);
    }
    __syncwarp();
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.lt.u32 p, %3, 2;\n\tsetp.ne.and.b32 q, %4, 0, p;\n\t"
        "@q cp.async.ca.shared.global [%0], [%1], 4;\n\tsetp.eq.and.b32 q, %4, 0, p;\n\t"
        "@q st.shared.f32 [%0], %2;\n\t}\n" ::"r"(scales + 4 * (lane & 1)),
        "l"((lane & 1 ? a.c.vscale : a.c.kscale) + ph), "f"(-1.f), "r"(lane), "r"((int)ok)
        : "memory");
  }

  // Scores, softmax and value product of 16 tokens of a stage.
  __device__ void tile(uint32_t st, const float2 sc, int t0, const Block& v, int lane) {
    if (sc.x < 0.f) return;   // not a page
    const int g = lane >> 2, qd = lane & 3;
    const bool full = t0 >= v.all_lo && t0 + 16 <= v.all_hi;
    // Two chains of matrix instructions: of the column groups, or of the halves of d.
    constexpr int C = R == 1 ? 2 : 1;
    float s[R][4], part[C][R][4];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[c][r][i] = 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const uint4 u0 = lds16(st + (koff[0] ^ (64 * c))), u1 = lds16(st + (koff[1] ^ (64 * c)));
      const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a0 = e4m3x2_to_f16x2(w0[i]), a1 = e4m3x2_to_f16x2(w1[i]);
        const uint32_t a2 = e4m3x2hi_to_f16x2(w0[i]), a3 = e4m3x2hi_to_f16x2(w1[i]);
#pragma unroll
        for (int r = 0; r < R; ++r) mma16816(part[i % C][r], a0, a1, a2, a3, qb[4 * c + i][r][0], qb[4 * c + i][r][1]);
      }
    }
    const bool zero_v = !(sc.y >= kLeastScale);
    const float w_page = zero_v ? kNoValue : sc.y, lw = __log2f(w_page), iw = __fdividef(1.f, w_page);
    // Weights under the reference as it is.  It stays while they are below
    // 2^14 (binary16 ends at 2^16).
    float y[R][4], most = 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float f0 = qf[r][0] * sc.x, f1 = qf[r][1] * sc.x, o0 = lw - m[r][0], o1 = lw - m[r][1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[r][i] = C == 2 ? part[0][r][i] + part[C - 1][r][i] : part[0][r][i];
        y[r][i] = ex2(fmaf(s[r][i], i & 1 ? f1 : f0, i & 1 ? o1 : o0));
        most = fmaxf(most, y[r][i]);
      }
    }
    if (!begun || !full || __any_sync(0xffffffffu, most > 16384.f)) {
      begun = true;
      const int t = t0 + token_of<D>(g);
#pragma unroll
      for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool in0 = t >= clo[r][i] && t < chi[r][i], in1 = t + 8 >= clo[r][i] && t + 8 < chi[r][i];
          const float f = qf[r][i] * sc.x;
          const float x0 = in0 ? fmaf(s[r][i], f, lw) : -INFINITY, x1 = in1 ? fmaf(s[r][2 + i], f, lw) : -INFINITY;
          float mx = fmaxf(x0, x1);
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const float mn = fmaxf(m[r][i], mx - kBelow);
          const float k = mn == m[r][i] ? 1.f : ex2(m[r][i] - mn);
          m[r][i] = mn;
          l[r][i] *= k;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            o[j][r][i] *= k;
            o[j][r][2 + i] *= k;
          }
          y[r][i] = in0 ? ex2(x0 - mn) : 0.f;
          y[r][2 + i] = in1 ? ex2(x1 - mn) : 0.f;
        }
      }
    }
    uint32_t pb[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[r][i] = fmaf(y[r][i] + y[r][2 + i], iw, l[r][i]);
        const __half2 p = __floats2half2_rn(y[r][2 * i], y[r][2 * i + 1]);   // token g + 8 i, both heads
        // 8 tokens x 8 heads to 8 heads x 8 tokens.
        asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n"
                     : "=r"(pb[r][i])
                     : "r"(*reinterpret_cast<const uint32_t*>(&p)));
      }
    }
    if (zero_v) return;   // warp-uniform: the page has no values
    uint32_t w[4][D / 32];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t src = st + voff[r];
      if constexpr (D == 128) {
        const uint4 u = lds16(src);
        w[r][0] = u.x; w[r][1] = u.y; w[r][2] = u.z; w[r][3] = u.w;
      } else {
        const uint2 u = lds8(src);
        w[r][0] = u.x; w[r][1] = u.y;
      }
    }
    if (!full) {
      // What a masked token's place holds may be NaN: its weight of 0 is not enough.
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int tok = t0 + token_of<D>(2 * qd + (r & 1)) + 8 * (r >> 1);
        if (tok < v.lo || tok >= v.hi)
#pragma unroll
          for (int k = 0; k < D / 32; ++k) w[r][k] = 0u;
      }
    }
#pragma unroll
    for (int k = 0; k < D / 32; ++k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // Bytes 4 k + 2 i and + 1 of the tokens of k = 2 qd, 2 qd + 1 and 2 qd + 8, + 9 side by side.
        const uint32_t x = __byte_perm(w[0][k], w[1][k], i ? 0x7362 : 0x5140);
        const uint32_t z = __byte_perm(w[2][k], w[3][k], i ? 0x7362 : 0x5140);
        const uint32_t a0 = e4m3x2_to_f16x2(x), a1 = e4m3x2hi_to_f16x2(x);
        const uint32_t a2 = e4m3x2_to_f16x2(z), a3 = e4m3x2hi_to_f16x2(z);
#pragma unroll
        for (int r = 0; r < R; ++r) mma16816(o[2 * k + i][r], a0, a1, a2, a3, pb[r][0], pb[r][1]);
      }
  }

  // Sums of L over the eight lanes of a head.
  __device__ void close() {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) l[r][i] += __shfl_xor_sync(0xffffffffu, l[r][i], k);
  }

  __device__ void write_out(const Kv8AttnArgs& a, const Block& v, int h, int lane) const {
    const int g = lane >> 2, qd = lane & 3;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 8 * r + 2 * qd + i;
        if (c >= v.ntok * a.G) continue;
        const int64_t base = column(a, v, h, c) + g * (D / 8);
        const float f = l[r][i] == 0.f ? 0.f : 1.f / l[r][i];   // an empty row is 0
#pragma unroll
        for (int j = 0; j < NJ; ++j) store_out(a.out, a.dtype, base + 2 * j, o[j][r][i] * f, o[j][r][2 + i] * f);
      }
  }

  // The record in shared memory: O as [8 R][D] floats whose 16-byte pieces are
  // turned by record_turn, (M, L) as [8 R].
  __device__ void write_record(float* rec, float2* ml, int lane) const {
    const int g = lane >> 2, qd = lane & 3;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 8 * r + 2 * qd + i;
#pragma unroll
        for (int j = 0; j < NJ; j += 2)
          *reinterpret_cast<float4*>(rec + c * D + 4 * ((g * (D / 32) + j / 2) ^ record_turn<D>(c))) =
              make_float4(o[j][r][i], o[j][r][2 + i], o[j + 1][r][i], o[j + 1][r][2 + i]);
        if (g == 0) ml[c] = make_float2(m[r][i], l[r][i]);
      }
  }
};

// Workspace: the prefix of tile counts over sequences (times Hkv), then per
// CTA two partial records of `cols` columns: 0 goes on with what an earlier
// CTA began, 1 is begun here and goes on.
struct DecodeWs {
  size_t ml, part, total;
};
__host__ __device__ inline DecodeWs decode_ws(int B, int cols, int d, int64_t ctas) {
  DecodeWs w;
  w.ml = ((size_t)(B + 1) * 8 + 255) & ~(size_t)255;
  w.part = (w.ml + (size_t)ctas * 2 * cols * 8 + 255) & ~(size_t)255;
  w.total = w.part + (size_t)ctas * 2 * cols * d * 4;
  return w;
}

template <int D, int R, int S>
__global__ void __launch_bounds__(DEC_WARPS * 32, 1)
    k_kv8_decode(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, Kv8AttnArgs a) {
  using L = DecLayout<D, S>;
  constexpr int T = 16 * S;             // tokens of a stage
  constexpr int RS = (R + S - 1) / S;   // stages that a record takes
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (s_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ int64_t s_warp[DEC_WARPS];
  __shared__ float2 s_ml[DEC_WARPS][2][8 * R];
  __shared__ int s_flags[DEC_WARPS], s_pair[DEC_WARPS][2][3];   // (sequence, block, head) of the records
  int64_t* pre = reinterpret_cast<int64_t*>(smem + L::prefix);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char* ring = smem + warp * DEC_STAGES * stage_bytes<D, S>();
  const float2* scales = reinterpret_cast<const float2*>(smem + L::scales) + warp * DEC_STAGES;
  const uint32_t ring_s = s_addr(ring), scales_s = s_addr(scales), bar_s = s_addr(smem + L::bars) + warp * DEC_STAGES * 8;
  if (lane == 0) {
    for (int i = 0; i < DEC_STAGES; ++i) mbar_init(bar_s + 8 * i, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  const int rows = 8 * R / a.G;   // query rows of a block
  // Prefix of the tile counts.
  int64_t carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += DEC_WARPS * 32) {
    const int b = b0 + tid;
    int64_t n = 0;
    if (b < a.B) {
      int row0, count, start;
      seq_of(a, b, row0, count, start);
      for (int k = 0; k * rows < count; ++k) n += block_of(a, row0, count, start, k, rows).tiles(T);
      n *= a.c.Hkv;
    }
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t base = carry, all = carry;
#pragma unroll
    for (int w = 0; w < DEC_WARPS; ++w) {
      if (w < warp) base += s_warp[w];
      all += s_warp[w];
    }
    if (b < a.B) pre[b] = base + incl - n;
    carry = all;
    __syncthreads();
  }
  if (tid == 0) pre[a.B] = carry;
  __syncthreads();
  const int64_t total = carry, share = (total + gridDim.x - 1) / gridDim.x;   // tiles of a CTA
  const int64_t chunk = (share + DEC_WARPS - 1) / DEC_WARPS;                    // of a warp
  const DecodeWs W = decode_ws(a.B, 8 * R, D, gridDim.x);
  char* ws = static_cast<char*>(a.ws);
  if (blockIdx.x == 0)
    for (int b = tid; b <= a.B; b += DEC_WARPS * 32) reinterpret_cast<int64_t*>(ws)[b] = pre[b];
  // Blocks without tiles: their output is 0.
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    int row0, count, start;
    seq_of(a, b, row0, count, start);
    for (int k = 0; k * rows < count; ++k) {
      const Block v = block_of(a, row0, count, start, k, rows);
      if (v.tiles(T) > 0) continue;   // (later blocks may have none: windows that lie past the table)
      for (int i = tid; i < v.ntok * a.Hq * D / 2; i += DEC_WARPS * 32)
        store_out(a.out, a.dtype, (int64_t)v.row0 * a.Hq * D + 2 * i, 0.f, 0.f);
    }
  }

  const int64_t last = min(total, (blockIdx.x + 1) * share);
  int64_t at = blockIdx.x * share + warp * chunk;
  const int64_t end = min(last, at + chunk);
  int flags = 0;   // 1: record 0 is there, 2: and holds its pair's end, 4: record 1 is there
  int b = 0;
  if (at < end) {
    int x = 0, y = a.B;   // pre[x] <= at < pre[y]
    while (y - x > 1) {
      const int z = (x + y) >> 1;
      if (pre[z] <= at) x = z; else y = z;
    }
    b = x;
  }
  Attend<D, R, S> A;
  A.place(lane);
  const int per = a.c.bs / T;    // tiles per page
  int stages = DEC_STAGES;       // of the ring
  uint32_t phases = 0;           // parity of each stage's next phase
  bool fault = false;
  while (at < end && !fault) {
    while (pre[b + 1] <= at) ++b;
    int row0, seq_rows, start;
    seq_of(a, b, row0, seq_rows, start);
    int64_t off = at - pre[b];
    Block v = block_of(a, row0, seq_rows, start, 0, rows);
    int nt = v.tiles(T);
    int k = 0;
    while (off >= (int64_t)nt * a.c.Hkv) {
      off -= (int64_t)nt * a.c.Hkv;
      v = block_of(a, row0, seq_rows, start, ++k, rows);
      nt = v.tiles(T);
    }
    const int h = (int)(off / nt), first = (int)(off % nt);
    const int count = (int)min((int64_t)(nt - first), end - at);
    A.load_queries(a, v, h, lane);
    A.reset();
    const int32_t* table = a.c.table + (int64_t)b * a.c.max_blocks;
    int pg = (v.lo / T + first) / per, sub = (v.lo / T + first) % per;   // tile to copy next
    int32_t page = table[pg];
    int issued = 0, taken = 0, ps = 0, gs = 0;   // tiles, and their stages (the ring is empty here)
    auto issue_next = [&]() {
      if (issued < count) {
        const int32_t cur = page;
        const int slot = T * sub;
        if (++sub == per) {
          sub = 0;
          ++pg;
          if (issued + 1 < count) page = table[pg];
        }
        A.issue(a, &mk, &mv, ring_s + ps * stage_bytes<D, S>(), scales_s + 8 * ps, bar_s + 8 * ps, cur, h, slot, lane);
        if (++ps == stages) ps = 0;
        ++issued;
      }
      cp_commit();
    };
    auto arrived = [&](int tries) {
      const bool ok = kv8_wait(bar_s + 8 * gs, (phases >> gs) & 1, tries);
      phases ^= 1u << gs;
      if (++gs == stages) gs = 0;
      ++taken;
      return ok;
    };
    __syncwarp();
    for (int s = 1; s < stages; ++s) issue_next();
    int t0 = T * (v.lo / T + first);
    for (int i = 0; i < count; ++i, t0 += T) {
      __syncwarp();   // every lane is done with the stage that is refilled
      issue_next();
      if (stages == DEC_STAGES) cp_wait<DEC_STAGES - 1>(); else cp_wait<DEC_STAGES - RS - 1>();   // the tile's scales
      const int at_s = gs;
      if (!arrived(a.tries)) {
        fault = true;
        kv8_wait(bar_s + 8 * at_s, ((phases >> at_s) & 1) ^ 1, kKv8Tries);   // it may still come
        break;
      }
      __syncwarp();
#pragma unroll 1
      for (int k = 0; k < S; ++k)
        if (S == 1 || (t0 + 16 * k < v.hi && t0 + 16 * k + 16 > v.lo))
          A.tile(ring_s + at_s * stage_bytes<D, S>() + 16 * k * D, scales[at_s], t0 + 16 * k, v, lane);
    }
    if (fault) {   // a copy that did not come in time: wait for the others on their way, and report it
      while (taken < issued) arrived(kKv8Tries);
      if (lane == 0) atomicExch(&g_kv8_decode_fault, 1);
    }
    A.close();
    if (count == nt) {
      A.write_out(a, v, h, lane);
    } else {
      // Record 1 into the ring's first stages: this was the warp's last pair.
      // Record 0 into its last ones, which the ring then does without.
      const int slot = first > 0 ? 0 : 1;
      if (slot == 0) stages = DEC_STAGES - RS;
      __syncwarp();
      A.write_record(reinterpret_cast<float*>(ring + (slot ? 0 : DEC_STAGES - RS) * stage_bytes<D, S>()), s_ml[warp][slot], lane);
      flags |= slot ? 4 : first + count == nt ? 3 : 1;
      if (lane == 0) {
        s_pair[warp][slot][0] = b;
        s_pair[warp][slot][1] = k;
        s_pair[warp][slot][2] = h;
      }
    }
    at += count;
  }
  cp_wait<0>();
  if (lane == 0) s_flags[warp] = flags;
  __syncthreads();
  // ---- join the parts of each pair: a record 1, or the first warp's record 0,
  // then the record 0 of the warps after it up to the pair's end ---------------
  for (int c = -1; c < DEC_WARPS; ++c) {
    if (!(c < 0 ? s_flags[0] & 1 : s_flags[c] & 4)) continue;
    int n = c < 0 ? 0 : 1, w = c + 1;   // records, the next warp
    bool closed = false;
    while (w < DEC_WARPS && !closed && (s_flags[w] & 1)) {
      closed = s_flags[w] & 2;
      ++w;
      ++n;
    }
    const int w0 = max(c, 0), s0 = c < 0 ? 0 : 1;
    const int pb = s_pair[w0][s0][0], pk = s_pair[w0][s0][1], ph = s_pair[w0][s0][2];
    int row0, count, start;
    seq_of(a, pb, row0, count, start);
    const Block v = block_of(a, row0, count, start, pk, rows);
    for (int i = tid; i < v.ntok * a.G * (D / 4); i += DEC_WARPS * 32) {
      const int col = i / (D / 4), f = i % (D / 4);
      float m = -INFINITY, l = 0.f;
      for (int k = 0; k < n; ++k) {
        const float2 u = s_ml[w0 + k][k == 0 ? s0 : 0][col];
        if (u.y != 0.f) m = fmaxf(m, u.x);   // a part without tokens has no O
      }
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < n; ++k) {
        const int s = k == 0 ? s0 : 0;
        const float2 u = s_ml[w0 + k][s][col];
        if (u.y == 0.f) continue;
        const float e = ex2(u.x - m);
        const float4 x = *reinterpret_cast<const float4*>(smem + ((w0 + k) * DEC_STAGES + (s ? 0 : DEC_STAGES - RS)) * stage_bytes<D, S>() +
                                                          4 * (col * D + 4 * (f ^ record_turn<D>(col))));
        l = fmaf(e, u.y, l);
        o.x = fmaf(e, x.x, o.x);
        o.y = fmaf(e, x.y, o.y);
        o.z = fmaf(e, x.z, o.z);
        o.w = fmaf(e, x.w, o.w);
      }
      if (c >= 0 && closed) {
        const float k = l == 0.f ? 0.f : 1.f / l;
        const int64_t to = A.column(a, v, ph, col) + 4 * f;
        store_out(a.out, a.dtype, to, o.x * k, o.y * k);
        store_out(a.out, a.dtype, to + 2, o.z * k, o.w * k);
      } else {
        const int64_t rec = (2 * (int64_t)blockIdx.x + s0) * 8 * R + col;
        reinterpret_cast<float4*>(ws + W.part)[rec * (D / 4) + f] = o;
        if (f == 0) reinterpret_cast<float2*>(ws + W.ml)[rec] = make_float2(m, l);
      }
    }
  }
}

// out = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) L_i over the partial records
// of one (query row, head).  With one row per sequence a block takes a (row,
// head); with several, a column of the pair that crosses the end of a CTA's
// range and began in it, of which there are fewer.  Bound by latency: first all
// records' (M, L) at once, then their O with the weights at hand, the warps
// taking turns.
template <int D>
__global__ void __launch_bounds__(MERGE_THREADS) k_kv8_merge(Kv8AttnArgs a, int ctas, int cols, int T) {
  __shared__ float s_w[MERGE_THREADS];
  __shared__ float s_red[2][MERGE_THREADS / 32];
  __shared__ float4 s_o[MERGE_THREADS];
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const char* ws = static_cast<const char*>(a.ws);
  const int64_t* pre = reinterpret_cast<const int64_t*>(ws);
  const int64_t total = pre[a.B], share = (total + ctas - 1) / ctas;
  const int rows = cols / a.G;
  int row, hq, col, nt;   // the output's row and head, its column, tiles of its pair
  int w0;                 // the CTA that began the pair
  int64_t x;              // the pair's first tile
  if (a.cu_q) {
    const int c = blockIdx.x / cols;
    col = blockIdx.x % cols;
    const int64_t cut = (c + 1) * share;
    for (int i = tid; i < a.B; i += MERGE_THREADS) {   // (loads that do not wait for the total)
      const int64_t lo = pre[i], hi = pre[i + 1];
      if (lo <= cut && cut < hi) s_b = i;
    }
    if (cut >= total) return;
    __syncthreads();
    int row0, count, start, k = 0;
    seq_of(a, s_b, row0, count, start);
    Block v = block_of(a, row0, count, start, 0, rows);
    nt = v.tiles(T);
    int64_t off = cut - pre[s_b];
    while (off >= (int64_t)nt * a.c.Hkv) {
      off -= (int64_t)nt * a.c.Hkv;
      v = block_of(a, row0, count, start, ++k, rows);
      nt = v.tiles(T);
    }
    const uint32_t h = (uint32_t)off / nt, first = (uint32_t)off - h * nt;   // off < nt Hkv <= 2^32
    x = cut - first;
    w0 = c;
    if (first == 0 || x < c * share || col >= v.ntok * a.G) return;
    row = v.row0 + col / a.G;
    hq = h * a.G + col % a.G;
  } else {
    row = blockIdx.x / a.Hq;
    hq = blockIdx.x % a.Hq;
    const int h = hq / a.G;
    col = hq % a.G;
    int row0, count, start;
    seq_of(a, row, row0, count, start);
    nt = block_of(a, row0, count, start, 0, rows).tiles(T);
    if (nt == 0) return;
    x = pre[row] + (int64_t)h * nt;
    w0 = (int)(x / share);
  }
  const int n = (int)((x + nt - 1) / share) - w0 + 1;
  if (n == 1) return;   // written by the CTA that held all of it
  const DecodeWs W = decode_ws(a.B, cols, D, ctas);
  const float2* ml = reinterpret_cast<const float2*>(ws + W.ml) + col;
  // Record of the i-th CTA: the first began the pair (record 1), the others go on with it.
  auto rec = [&](int i) { return (2 * (int64_t)(w0 + i) + (i == 0 ? 1 : 0)) * cols; };
  const float2 v = tid < n ? ml[rec(tid)] : make_float2(-INFINITY, 0.f);
  float m = v.y != 0.f ? v.x : -INFINITY;   // a part without tokens has no O
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) s_red[0][warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < MERGE_THREADS / 32; ++i) m = fmaxf(m, s_red[0][i]);
  const float e0 = v.y != 0.f ? ex2(v.x - m) : 0.f;
  s_w[tid] = e0;
  float l = e0 * v.y;
#pragma unroll
  for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (lane == 0) s_red[1][warp] = l;
  __syncthreads();
  constexpr int LPR = D / 4, ROWS = MERGE_THREADS / LPR;   // threads per record, records at a time
  const int r = tid / LPR, c = tid % LPR;
  const float4* part = reinterpret_cast<const float4*>(ws + W.part);
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = r; i < n; i += ROWS) {
    const float e = s_w[i];
    if (e == 0.f) continue;
    const float4 u = part[(rec(i) + col) * LPR + c];
    o.x = fmaf(e, u.x, o.x);
    o.y = fmaf(e, u.y, o.y);
    o.z = fmaf(e, u.z, o.z);
    o.w = fmaf(e, u.w, o.w);
  }
  s_o[tid] = o;
  __syncthreads();
  if (tid < LPR) {
    l = 0.f;
#pragma unroll
    for (int i = 0; i < MERGE_THREADS / 32; ++i) l += s_red[1][i];
#pragma unroll
    for (int i = 1; i < ROWS; ++i) {
      const float4 u = s_o[i * LPR + tid];
      o.x += u.x;
      o.y += u.y;
      o.z += u.z;
      o.w += u.w;
    }
    const float f = l == 0.f ? 0.f : 1.f / l;
    const int64_t at = ((int64_t)row * a.Hq + hq) * D + 4 * tid;
    store_out(a.out, a.dtype, at, o.x * f, o.y * f);
    store_out(a.out, a.dtype, at + 2, o.z * f, o.w * f);
  }
}

int decode_ctas(int sms) { return std::min(sms, MERGE_THREADS); }

// cuTensorMapEncodeTiled through the runtime's driver entry point (no link
// against the driver library).
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn find_encode() {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<EncodeTiledFn>(p);
}

// Codes as rows of 128 bytes (one token of d = 128, two of d = 64), in boxes of
// a stage's tokens.  Rows of 64 bytes took TMA as long as rows of 128.
bool make_map(CUtensorMap* map, const void* codes, int64_t tokens, int d, int box_tokens) {
  static const EncodeTiledFn fn = find_encode();
  if (!fn) return false;
  const int per = 128 / d;
  const cuuint64_t dims[2] = {128, (cuuint64_t)(tokens / per)};
  const cuuint64_t strides[1] = {128};
  const cuuint32_t box[2] = {128, (cuuint32_t)(box_tokens / per)};
  const cuuint32_t es[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int R, int S>
cudaError_t run_decode(const Kv8AttnArgs& a, int sms, cudaStream_t s) {
  if (a.c.bs % (16 * S) != 0) return cudaErrorInvalidValue;   // a stage would cross pages
  const int64_t rows = a.c.num_blocks * a.c.Hkv * a.c.bs;
  CUtensorMap mk, mv;
  if (!make_map(&mk, a.c.kcodes, rows, D, 16 * S) || !make_map(&mv, a.c.vcodes, rows, D, 16 * S)) return cudaErrorInvalidValue;
  const int smem = DecLayout<D, S>::total(a.B);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_kv8_decode<D, R, S>, DecLayout<D, S>::total(kKv8MaxSeqs), done);
  if (e != cudaSuccess) return e;
  k_kv8_decode<D, R, S><<<sms, DEC_WARPS * 32, smem, s>>>(mk, mv, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const unsigned blocks = a.cu_q ? sms * 8 * R : (unsigned)(a.n * a.Hq);
  k_kv8_merge<D><<<blocks, MERGE_THREADS, 0, s>>>(a, sms, 8 * R, 16 * S);
  return cudaGetLastError();
}

}  // namespace

size_t kv8_decode_workspace(int B, int d, int sms) {
  return decode_ws(B, 16, d, decode_ctas(sms)).total;
}

// The smaller matrix products where the rows of a sequence (on average, and
// all of them in a decode) fit into 8 columns: 16 x 32768 tokens and groups of
// four 195 us against 214 us with 16, 16 x 2 rows 47 us against 56 us.  An average
// above the `most` rows that a sequence may have here is that of others, beside
// which single rows are the common case: the smaller ones too.  With d = 64 a
// stage holds 32 tokens where pages hold whole stages: half as many copies to
// issue, and 16 x 32768 tokens take 104 us against 122 us with 16 tokens a stage,
// the ragged sequences 52 us against 56 us, 64 x 300 tokens 23.7 us against 24.9 us.
cudaError_t launch_kv8_decode(const Kv8AttnArgs& a, int sms, cudaStream_t s) {
  sms = decode_ctas(sms);
  const bool wide = a.G > 8 || (a.n * a.G > 8 * (int64_t)a.B && a.n <= a.most * (int64_t)a.B);
  if (a.d == 128) return wide ? run_decode<128, 2, 1>(a, sms, s) : run_decode<128, 1, 1>(a, sms, s);
  if (a.c.bs % 32 == 0) return wide ? run_decode<64, 2, 2>(a, sms, s) : run_decode<64, 1, 2>(a, sms, s);
  return wide ? run_decode<64, 2, 1>(a, sms, s) : run_decode<64, 1, 1>(a, sms, s);
}

cudaError_t read_and_clear_kv8_decode_fault(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_kv8_decode_fault, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_kv8_decode_fault, &zero, sizeof(int));
}

}  // namespace tqk
