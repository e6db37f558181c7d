// Prompt attention over the 8-bit paged KV cache on the 5th-generation tensor
// cores (tcgen05, sm_100a): ragged batches of rows, causal, optional window.
//
// The mathematics is that of the decode kernel: with x_t = scale log2(e) a_t
// <q, k_t> for key code k_t and page scale a_t, value page scale w_t and M a
// reference near the maximum of x_t + log2(w_t),
//   O = sum_t 2^(x_t + log2 w_t - M) v_t,   L = sum_t 2^(x_t + log2 w_t - M) / w_t,
//   out = O / L.
// Both products run in binary16 with fp32 accumulation: codes and (scaled by
// a power of two per row) queries are exact in it, the weights are rounded to
// it once.  The page scales enter as one factor and one summand per 16
// tokens, so a score costs one fused multiply-add and one exponential; M
// is 2^6 below the maximum when it is set and stays until a sum of 16 weights
// leaves binary16, so the common half takes no maximum.
//
// A work item is a kv head and 2 x 128 packed rows: row r of a tile is token
// r / G, head r % G of the group, so the G query heads that share a kv head
// share its keys.  Roles of a CTA (one per SM):
//   warps 0-3, 4-7  softmax of tile 0 / tile 1, one row per thread: scores from
//                   tensor memory, weights back to tensor memory (as the A
//                   operand of the value product, over the scores' columns),
//                   rescaling of O only when a weight passes 2^12;
//   warps 8-11      converters: 8-bit pages to binary16 operands in shared
//                   memory (128-byte swizzle), the next codes on their way by
//                   cp.async (each lane copies what it converts);
//   warps 12, 13    issue the MMAs of tile 0 / tile 1: S = Q K^T, O += P V.
// A step of 128 tokens is taken in two halves of 64 with a place each for
// their scores: one half's products run while the other is in its softmax.
// The 128-token steps of all items form one list that the CTAs share in equal
// contiguous ranges (few rows over long contexts split, ragged batches
// balance); an item that is cut leaves (O, M, L) per part for k_kv8_join.
//
// Bound by the softmax warps' latency: a half takes about 2000 cycles at 50%
// of the issue slots, the tensor pipes are 43% busy (the products alone would
// take 1300 at the shared-memory rate of their 64-column operands, which read
// the queries twice a step).  Measured on a B200 (device time, in a short run at
// 1965 MHz, and in a long one, where the power limit takes the clock to 1830 to
// 1860 MHz): 8192 rows, 32 heads over 8, d = 128: 571 and 610 us, 960 and 900
// TFLOP/s; 2033 rows of two chunks over 16384 cached: 514 and 563 us, 1030 and
// 950; ragged rows of d = 64 under a window of 1024: 101 and 99 us.  What was tried and measured no
// faster (8192 rows): one half after the other with a maximum each 883 us; a
// quarter of the exponentials as polynomials 644 us; turns for the
// exponentials of the two tiles 677 us; two threads per row 760 us; unrolled
// careful halves 581 us (the roles' code has to stay in the instruction
// caches: unrolled loops cost threefold at first).
//
// Every mbarrier wait is bounded; on expiry the kernel records a fault,
// drains its MMAs, frees its tensor memory and returns.
#include "tq_internal.h"
#include "tq_kv8.cuh"
#include "tq_tc_common.cuh"

namespace tqk {

__device__ int g_kv8_fault = 0;

namespace {

constexpr int PF_THREADS = 512;               // warps 14, 15 idle: registers move by warpgroup
// Registers per thread of the softmax, converter and MMA warpgroups: 2 * 168 +
// 104 + 72 = 4 * 128, what the block is launched with.
constexpr int PF_REGS_S = 168, PF_REGS_C = 104, PF_REGS_M = 72;
constexpr int PF_TILE = 128;                  // tokens per step, rows per tile
// What an item costs besides its steps, in steps: 8192 rows take 622, 568, 570
// and 575 us with 3, 4, 5 and 6.
constexpr int kItemCost = 4;
// Rows x heads of a group up to which the decode kernel takes a sequence: over
// 5000 cached tokens (16 sequences) it takes 47, 61, 93 and 97 us for 8, 16, 24
// and 32, this one 92 to 93 us.
constexpr int kNarrow = 16;
// Below these a call over both kinds of sequences is not split (launch_kv8_prefill).
constexpr int kFewTiles = 25000, kMixed = 4000;
// M is set kBelow below a maximum (log2), so the largest weight is at least 2^6
// and binary16 takes weights down to 2^-31 of it, of which a long tail may be
// made.  M is set anew, and O rescaled, when a weight passes 2^kLazy; 16 weights
// may sum to kMostSum before their maximum is looked at: a larger sum holds a
// weight of nearly 2^kLazy at least, and what is below it fits binary16.  8192
// rows take 570 us with kBelow 0 (kLazy 8, sums to 2^14), 5 and 6, and 578 us with
// 8, where the reference moves too often; rows under a window 107, 104, 105 and
// 109 us.
constexpr float kBelow = 6.f;
constexpr float kLazy = 12.f;
constexpr float kMostSum = 65504.f;

// Shared memory above a 1024-byte aligned base: V and K stages, Q tiles (all
// in halves of 64 columns, 128 rows of 128 bytes), then small records.
template <int D>
struct PfLayout {
  static constexpr uint32_t kHalf = 128 * 128;
  static constexpr uint32_t kTile = kHalf * (D / 64);
  static constexpr uint32_t V = 0, K = 2 * kTile, Q = 4 * kTile;
  static constexpr uint32_t RAW = 6 * kTile;            // codes of the next K and V step, as they are in the pages
  static constexpr uint32_t kRaw = 128 * D;
  static constexpr uint32_t SC = RAW + 2 * kRaw;        // float4 [4 slots][8 groups]: (a, log2 w, 1 / w, -)
  static constexpr uint32_t QF = SC + 4 * 8 * 16;       // float [256]: row factors
  static constexpr uint32_t BAR = QF + 256 * 4;         // barriers
  static constexpr uint32_t MISC = BAR + 32 * 8;
  static constexpr uint32_t total = MISC + 256 + 1024;  // + alignment slack
};
// Barriers; B_S (scores there), B_P (weights there) and B_O (value product
// done): tile x, half h at 2 x + h.  A wait names the phase by its parity, so a
// waiter has to know that the phase before it is complete and that the one
// after it cannot be.
enum { B_KF = 0, B_KE = 2, B_VF = 4, B_VE = 6, B_SC = 8, B_S = 12, B_P = 16, B_Q = 20, B_O = 22, B_DONE = 26 };

// Rows, tokens and steps of item (b, qt): the same for every kv head.
struct Item {
  int row0, ntok, pos0;     // first row, tokens (up to 2 * TPT), position of the first
  int a[2], e[2];           // steps [a, e) of each tile; a = e where the tile has no rows
  int lo, hi;               // tokens that any row sees
  __device__ int steps() const { return max(e[0], e[1]) - a[0]; }
};

__device__ __forceinline__ Item item_of(const Kv8AttnArgs& a, int row0, int count, int start, int qt, int TPT) {
  Item it;
  const int t0 = qt * 2 * TPT;
  const int cap = a.c.max_blocks * a.c.bs;
  it.row0 = row0 + t0;
  it.ntok = min(count - t0, 2 * TPT);
  it.pos0 = start + t0;
  it.lo = it.hi = 0;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int n = min(it.ntok - x * TPT, TPT);
    it.a[x] = it.e[x] = 0;
    if (n > 0) {
      const int p = it.pos0 + x * TPT;
      const int hi = min(max(p + n, 0), cap);
      const int lo = a.window > 0 ? min(max(p - a.window + 1, 0), hi) : 0;
      it.a[x] = lo / PF_TILE;
      it.e[x] = max((hi + PF_TILE - 1) / PF_TILE, it.a[x] + 1);   // a step even where nothing is seen
      if (x == 0) it.lo = lo;
      it.hi = hi;
    }
  }
  return it;
}

// The CTA's walk over its range of steps.
struct Walk {
  int b, qt, h, off;        // next item and its first unit
  int64_t left;             // units left
  int row0, count, start;   // of sequence b
  Item it;                  // of the current part
  int ib, iqt, ih;
  int j0, j1;               // its steps
  bool begun, ended;        // it holds the item's first / last step
  // The next part, if any.  An item is kItemCost units for its start, then one
  // per step.
  __device__ bool next(const Kv8AttnArgs& a, int TPT) {
    while (left > 0) {
      while (qt * 2 * TPT >= count) {   // the next sequence that has rows
        if (++b >= a.B) return false;
        qt = 0;
        ragged_seq(a, b, row0, count, start);
      }
      it = item_of(a, row0, count, start, qt, TPT);
      const int n = it.steps(), to = (int)min((int64_t)(n + kItemCost), off + left);
      const int s0 = max(off - kItemCost, 0), s1 = max(to - kItemCost, 0);
      j0 = it.a[0] + s0;
      j1 = it.a[0] + s1;
      begun = s0 == 0;
      ended = s1 == n;
      left -= to - off;
      ib = b;
      iqt = qt;
      ih = h;
      off = 0;
      if (++h == a.c.Hkv) {
        h = 0;
        ++qt;
      }
      if (s0 < s1) return true;
    }
    return false;
  }
};

struct JoinHead {
  int valid, last, b, qt, h, pad[3];
};
struct PfWs {
  size_t ml, part, total;
};
__host__ __device__ inline PfWs pf_ws(int d, int64_t ctas) {
  PfWs w;
  w.ml = ((size_t)ctas * 2 * sizeof(JoinHead) + 255) & ~(size_t)255;
  w.part = w.ml + (size_t)ctas * 2 * 256 * 8;
  w.total = w.part + (size_t)ctas * 2 * 256 * d * 4;
  return w;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\t"
      "mov.b64 {%0, %1}, x;\n\t}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// kv8_wait for the converters, which run ahead: their polls leave the issue
// slots to the softmax warps.
__device__ __forceinline__ bool lazy_wait(uint32_t bar, uint32_t parity, int tries) {
  for (int it = 0; it < tries; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    __nanosleep(128);
  }
  return false;
}

// ---- tensor memory ----------------------------------------------------------
// Loads wait for their data in the same statement: nothing may read the
// registers before.
// 16 columns of the thread's lane.
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15"
      "}, [%16];\n\ttcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(addr)
      : "memory");
}
// 32 columns of the thread's lane.
__device__ __forceinline__ void tm_ld32(uint32_t addr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31"
      "}, [%32];\n\ttcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr)
      : "memory");
}
// 64 columns of the thread's lane.
__device__ __forceinline__ void tm_ld64(uint32_t addr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%64];\n\ttcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
        "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
        "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]),
        "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]), "=r"(r[41]), "=r"(r[42]),
        "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]), "=r"(r[49]),
        "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
        "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8"
      "};\n" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16"
      "};\n" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {"
      "%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32"
      "};\n" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
        "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
        "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }

// B operand whose N axis is contiguous: rows are K (tokens) of 128 bytes (64
// columns, 128-byte swizzle), 1024 bytes between groups of 8 rows, `lbo`
// bytes between halves of 64 columns.
__device__ __forceinline__ uint64_t v_desc(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// S = Q K^T for 64 tokens, then an arrival on `bar` when it is done.
template <int D>
__device__ __forceinline__ void mma_scores(uint32_t d, uint64_t q, uint64_t k, uint32_t bar) {
  constexpr uint32_t ID = tc_idesc_f16(64);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    const uint64_t o = (uint64_t)((i / 4) * (PfLayout<D>::kHalf >> 4) + 2 * (i % 4));
    tc_mma_f16(d, q + o, k + o, ID, i > 0);
  }
  tc_commit(bar);
}

// O (+)= P V for 64 tokens: A in tensor memory (lane = row), B in shared memory.
template <int D>
__device__ __forceinline__ void mma_values(uint32_t d, uint32_t p, uint64_t v, uint32_t acc, uint32_t bar) {
  constexpr uint32_t ID = tc_idesc_f16(D) | (1u << 16);   // B with its N axis contiguous
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t}\n" ::"r"(d),
        "r"(p + 8 * i), "l"(v + (uint64_t)(i * 2048 >> 4)), "r"(i ? 1u : acc), "r"(ID));
  tc_commit(bar);
}

// ---- converters ----------------------------------------------------------------
// Four codes to binary16 (times 1).
__device__ __forceinline__ void cvt_e4m3x4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// The two groups of 16 tokens that a converter warp takes of one step.
struct Groups {
  int t, lo, hi;      // first token, tokens that count
  int32_t q0, q1;     // pages, -1 where nothing is to be read
  int64_t h0, h1;     // (page, head) records
  int s0, s1;         // slots
  __device__ void find(const Kv8AttnArgs& a, const Walk& wk, int j, int cw) {
    const int32_t* table = a.c.table + (int64_t)wk.ib * a.c.max_blocks;
    t = j * PF_TILE + 32 * cw;
    lo = wk.it.lo;
    hi = wk.it.hi;
    const int p0 = t / a.c.bs, p1 = (t + 16) / a.c.bs;
    s0 = t - p0 * a.c.bs;
    s1 = t + 16 - p1 * a.c.bs;
    q0 = t < hi && t + 16 > lo ? __ldg(table + p0) : -1;
    q1 = t + 16 < hi && t + 32 > lo ? __ldg(table + p1) : -1;
    head = wk.ih;
  }
  int head;
  __device__ void place(const Kv8AttnArgs& a) {
    if (q0 >= a.c.num_blocks) q0 = -1;
    if (q1 >= a.c.num_blocks) q1 = -1;
    h0 = (int64_t)max(q0, 0) * a.c.Hkv + head;
    h1 = (int64_t)max(q1, 0) * a.c.Hkv + head;
  }
};

// A warp takes rows (tokens) 32 w .. 32 w + 31 of a tile: D / 16 lanes per
// row, 16 codes each.  A lane copies the pieces that it will convert.
template <int D>
struct Codes {
  static constexpr int LPR = D / 16, RPL = 32 / LPR, N = 32 / RPL;   // lanes per row, rows per round, rounds
  __device__ static void copy(uint32_t raw, const uint8_t* codes, const Groups& g, int bs, int warp, int lane) {
    const int64_t at = (lane / LPR) * D + (lane % LPR) * 16;
    const uint8_t* p0 = codes + (g.h0 * bs + g.s0) * D + at;
    const uint8_t* p1 = codes + (g.h1 * bs + g.s1) * D + at;
    uint32_t dst = raw + warp * 32 * D + lane * 16;
    int t = g.t + lane / LPR;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool second = i >= N / 2;
      const int bytes = (second ? g.q1 : g.q0) >= 0 && t >= g.lo && t < g.hi ? 16 : 0;   // else zeros
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst),
                   "l"((second ? p1 : p0) + (second ? i - N / 2 : i) * RPL * D), "r"(bytes)
                   : "memory");
      dst += 512;
      t += RPL;
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  }
  // tile: shared address of row 0 of the tile; rows of 128 bytes, chunk c of
  // 16 bytes at c ^ (row & 7).  Lanes of the upper half store their second
  // chunk first: the eight lanes of a phase then hit eight different chunks.
  // z0, z1: store zeros for the group.
  template <bool VALUES>
  __device__ static void convert(uint32_t tile, const unsigned char* raw, int warp, int lane, bool z0, bool z1) {
    const int piece = lane % LPR, half = piece / 4, c0 = 2 * (piece % 4) + half, c1 = c0 ^ 1;
    const unsigned char* src = raw + warp * 32 * D + lane * 16;
    const int o0 = 8 * half, o1 = 8 - o0;
    tile += half * PfLayout<D>::kHalf;
#pragma unroll 2
    for (int i = 0; i < N; ++i) {
      const int row = 32 * warp + i * RPL + lane / LPR;
      const uint32_t base = tile + row * 128;
      uint2 u = *reinterpret_cast<const uint2*>(src + 512 * i + o0), v = *reinterpret_cast<const uint2*>(src + 512 * i + o1);
      if (VALUES && (i < N / 2 ? z0 : z1)) u = v = make_uint2(0, 0);
      uint32_t f[8];
      cvt_e4m3x4(u.x, f[0], f[1]);
      cvt_e4m3x4(u.y, f[2], f[3]);
      cvt_e4m3x4(v.x, f[4], f[5]);
      cvt_e4m3x4(v.y, f[6], f[7]);
      sts128(base + ((c0 ^ (row & 7)) << 4), f[0], f[1], f[2], f[3]);
      sts128(base + ((c1 ^ (row & 7)) << 4), f[4], f[5], f[6], f[7]);
    }
  }
};
// ---- queries ----------------------------------------------------------------
// A warp's 32 rows of a tile, in two turns: the rows as they are to the tile's
// place (asynchronously, once its scores are done with the last item's), then
// in place to binary16 scaled by a power of two per row; factors scale
// log2(e) / 2^e to qf.  Each lane converts what it has copied.
template <int D>
struct Queries {
  static constexpr int LPR = D / 8, RPL = 32 / LPR, N = 32 / RPL;   // lanes per row (16 bytes each), rows per round
  __device__ static uint32_t place(uint32_t tile, int row, int piece) {
    return tile + (piece / 8) * PfLayout<D>::kHalf + row * 128 + (((piece % 8) ^ (row & 7)) << 4);
  }
  // row0, ntok: the tile's first row and tokens.  invG: 65536 / G + 1.
  __device__ static void copy(const Kv8AttnArgs& a, int row0, int ntok, int h, uint32_t invG, uint32_t tile, int warp4,
                              int lane) {
    const int piece = lane % LPR, rows = ntok * a.G;
    const uint16_t* q = static_cast<const uint16_t*>(a.q) + ((int64_t)row0 * a.Hq + (int64_t)h * a.G) * D + piece * 8;
#pragma unroll 2
    for (int i = 0; i < N; ++i) {
      const int row = 32 * warp4 + i * RPL + lane / LPR;
      const int tok = (int)((row * invG) >> 16);       // row / G, exact for row < 128
      const bool in = row < rows;
      const uint16_t* src = in ? q + ((int64_t)tok * a.Hq + (row - tok * a.G)) * D : q;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(place(tile, row, piece)), "l"(src),
                   "r"(in ? 16 : 0)
                   : "memory");
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
  }
  __device__ static void convert(const Kv8AttnArgs& a, uint32_t tile, float* qf, int warp4, int lane) {
    const int piece = lane % LPR;
    if (a.dtype == TQ_F16) {   // as it is
      qf[32 * warp4 + lane] = a.scale_log2;
      return;
    }
    // Four rounds at a time, stage by stage: their latencies overlap.
#pragma unroll 1
    for (int i = 0; i < N; i += 4) {
      const int row = 32 * warp4 + i * RPL + lane / LPR;   // and RPL on, for each round
      uint32_t w[4][4], mx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(w[j][0]), "=r"(w[j][1]), "=r"(w[j][2]), "=r"(w[j][3])
                     : "r"(place(tile, row + j * RPL, piece))
                     : "memory");
      // Magnitudes of bf16 order like their bits; only the exponent counts.
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) m = max(m, max(w[j][k] & 0x7FFF0000u, (w[j][k] << 16) & 0x7FFF0000u));
        mx[j] = m;
      }
#pragma unroll
      for (int o = 1; o < LPR; o <<= 1)
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = max(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], o));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // 2^e that takes the largest to [2^14, 2^15), in two factors that fp32 can hold.
        const int e = mx[j] ? 14 + 127 - min(max((int)(mx[j] >> 23), 1), 254) : 0;
        const int e1 = e / 2, e2 = e - e1;
        const float f1 = __uint_as_float((uint32_t)(127 + e1) << 23), f2 = __uint_as_float((uint32_t)(127 + e2) << 23);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __half2 hh = __floats2half2_rn(__uint_as_float(w[j][k] << 16) * f1 * f2,
                                               __uint_as_float(w[j][k] & 0xFFFF0000u) * f1 * f2);
          w[j][k] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        sts128(place(tile, row + j * RPL, piece), w[j][0], w[j][1], w[j][2], w[j][3]);
        if (piece == 0)
          qf[row + j * RPL] =
              a.scale_log2 * __uint_as_float((uint32_t)(127 - e1) << 23) * __uint_as_float((uint32_t)(127 - e2) << 23);
      }
    }
  }
};

// Pieces p[0..3] of the lane's row become piece (lane % 4) of the four rows of
// its group of four lanes: a store of one piece per lane then covers 64
// contiguous bytes of eight rows, not 16 bytes of thirty-two.
__device__ __forceinline__ void turn4(uint4 (&p)[4], int lane) {
  auto trade = [&](uint4& x, uint4& y, bool odd, int o) {   // odd lanes give x, even ones y
    const uint4 s = odd ? x : y;
    uint4 r;
    r.x = __shfl_xor_sync(0xffffffffu, s.x, o);
    r.y = __shfl_xor_sync(0xffffffffu, s.y, o);
    r.z = __shfl_xor_sync(0xffffffffu, s.z, o);
    r.w = __shfl_xor_sync(0xffffffffu, s.w, o);
    if (odd) x = r; else y = r;
  };
  trade(p[0], p[1], lane & 1, 1);
  trade(p[2], p[3], lane & 1, 1);
  trade(p[0], p[2], lane & 2, 2);
  trade(p[1], p[3], lane & 2, 2);
}

template <int D>
__global__ void __launch_bounds__(PF_THREADS, 1) k_kv8_prefill(Kv8AttnArgs a) {
  using L = PfLayout<D>;
  extern __shared__ unsigned char smem_raw[];
  const uint32_t raw_s = (uint32_t)__cvta_generic_to_shared(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  unsigned char* base = smem_raw + (base_s - raw_s);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar = base_s + L::BAR;
  auto bar_at = [&](int i) { return bar + 8 * i; };
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(base + L::MISC);
  int* s_start = reinterpret_cast<int*>(base + L::MISC + 16);          // b, qt, h, off
  int64_t* s_sum = reinterpret_cast<int64_t*>(base + L::MISC + 64);    // [16]
  const int TPT = PF_TILE / a.G;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_at(B_KF + i), 4);
      mbar_init(bar_at(B_KE + i), 2);
      mbar_init(bar_at(B_VF + i), 4);
      mbar_init(bar_at(B_VE + i), 2);
      mbar_init(bar_at(B_Q + i), 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar_at(B_SC + i), 4);
      mbar_init(bar_at(B_S + i), 1);
      mbar_init(bar_at(B_P + i), 4);
      mbar_init(bar_at(B_O + i), 1);
    }
    mbar_init(bar_at(B_DONE), 2);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 12) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                     (uint32_t)__cvta_generic_to_shared(s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  // ---- plan: steps of every sequence, the CTA's range, its first item ---------
  int64_t* steps = reinterpret_cast<int64_t*>(base);   // [B], in the operands' space
  for (int b = warp; b < a.B; b += PF_THREADS / 32) {
    int row0, count, start;
    ragged_seq(a, b, row0, count, start);
    const int nq = (count + 2 * TPT - 1) / (2 * TPT);
    int64_t n = 0;
    for (int q = lane; q < nq; q += 32) n += item_of(a, row0, count, start, q, TPT).steps() + kItemCost;
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (lane == 0) steps[b] = n * a.c.Hkv;
  }
  __syncthreads();
  int64_t sum = 0;
  for (int b = tid; b < a.B; b += PF_THREADS) sum += steps[b];
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < PF_THREADS / 32; ++w) total += s_sum[w];
  const int64_t at = total / gridDim.x * blockIdx.x + min((int64_t)blockIdx.x, total % gridDim.x);
  const int64_t mine = total / gridDim.x + (blockIdx.x < total % gridDim.x ? 1 : 0);
  if (warp == 0 && mine > 0) {
    int64_t before = 0;
    int b = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {      // the sequence that holds unit `at`
      const int64_t v = b0 + lane < a.B ? steps[b0 + lane] : 0;
      int64_t incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, before + incl > at);
      if (in) {
        const int f = __ffs(in) - 1;
        b = b0 + f;
        before += __shfl_sync(0xffffffffu, incl - v, f);
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    int row0, count, start;
    ragged_seq(a, b, row0, count, start);
    const int nq = (count + 2 * TPT - 1) / (2 * TPT);
    for (int q0 = 0; q0 < nq; q0 += 32) {
      const int n = q0 + lane < nq ? item_of(a, row0, count, start, q0 + lane, TPT).steps() + kItemCost : 0;
      const int64_t v = (int64_t)n * a.c.Hkv;
      int64_t incl = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += u;
      }
      const uint32_t in = __ballot_sync(0xffffffffu, before + incl > at);
      if (in) {
        const int f = __ffs(in) - 1;
        if (lane == f) {
          const int64_t off = at - (before + incl - v);
          s_start[0] = b;
          s_start[1] = q0 + lane;
          s_start[2] = (int)(off / n);
          s_start[3] = (int)(off % n);
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = *s_tmem;
  Walk wk;
  wk.b = s_start[0];
  wk.qt = s_start[1];
  wk.h = s_start[2];
  wk.off = s_start[3];
  wk.left = mine;
  if (mine > 0) ragged_seq(a, wk.b, wk.row0, wk.count, wk.start);
  const PfWs W = pf_ws(D, gridDim.x);
  char* ws = static_cast<char*>(a.ws);
  JoinHead* heads = reinterpret_cast<JoinHead*>(ws) + 2 * blockIdx.x;
  bool fault = false;

  if (warp >= 8 && warp < 12) {
    // ---- converters -------------------------------------------------------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(PF_REGS_C));
    const int cw = warp - 8;
    uint32_t c = 0;                 // steps converted
    const uint32_t raw = base_s + L::RAW;
    Groups now{}, then{};           // the step whose codes are on their way, the next one
    float ka = 0.f, w0 = 0.f, w1 = 0.f;
    bool has_page = false;
    auto scales = [&]() {
      has_page = (lane ? now.q1 : now.q0) >= 0;
      ka = has_page ? __ldg(a.c.kscale + (lane ? now.h1 : now.h0)) : 0.f;
      w0 = now.q0 >= 0 ? __ldg(a.c.vscale + now.h0) : 0.f;
      w1 = now.q1 >= 0 ? __ldg(a.c.vscale + now.h1) : 0.f;
    };
    bool more = wk.next(a, TPT);    // step j of the walk is `then`
    int j = more ? wk.j0 : 0;
    auto advance = [&]() {
      if (++j >= wk.j1) {
        more = wk.next(a, TPT);
        j = wk.j0;
      }
      if (more) then.find(a, wk, j, cw);
    };
    if (more) {
      now.find(a, wk, j, cw);
      now.place(a);
      Codes<D>::copy(raw, a.c.kcodes, now, a.c.bs, cw, lane);
      Codes<D>::copy(raw + L::kRaw, a.c.vcodes, now, a.c.bs, cw, lane);
      scales();
      bool has = true;
      advance();
      while (has) {
        const uint32_t st = c & 1, par = (c >> 1) & 1;
        // Values of a page without a scale are 0 whatever its codes.
        const bool z0 = !(w0 >= kLeastScale), z1 = !(w1 >= kLeastScale);
        cp_wait<1>();   // the lane's key codes
        if (c >= 2 && !lazy_wait(bar_at(B_KE + st), par ^ 1, a.tries)) { fault = true; break; }
        if (lane < 2) {
          const float vw = (lane ? z1 : z0) ? kNoValue : lane ? w1 : w0;
          reinterpret_cast<float4*>(base + L::SC)[(c & 3) * 8 + 2 * cw + lane] =
              make_float4(ka, has_page ? __log2f(vw) : -INFINITY, 1.f / vw, 0.f);   // no page: weights of 0
        }
        Codes<D>::template convert<false>(base_s + L::K + st * L::kTile, base + L::RAW, cw, lane, false, false);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar_at(B_SC + (c & 3)));
          mbar_arrive(bar_at(B_KF + st));
        }
        if (more) {
          now = then;
          now.place(a);
          Codes<D>::copy(raw, a.c.kcodes, now, a.c.bs, cw, lane);
          scales();
          cp_wait<1>();
        } else {
          cp_wait<0>();
        }
        if (c >= 2 && !lazy_wait(bar_at(B_VE + st), par ^ 1, a.tries)) { fault = true; break; }
        Codes<D>::template convert<true>(base_s + L::V + st * L::kTile, base + L::RAW + L::kRaw, cw, lane, z0, z1);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_at(B_VF + st));
        has = more;
        if (more) {
          Codes<D>::copy(raw + L::kRaw, a.c.vcodes, now, a.c.bs, cw, lane);
          advance();
        }
        ++c;
      }
      cp_wait<0>();
    }
  } else if (warp >= 12) {
    // ---- MMA issue ----------------------------------------------------------------
    // The whole warp runs the loop and one elected lane issues: under a branch
    // on the lane number each MMA cost about 100 cycles to issue.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(PF_REGS_M));
    if (warp < 14) {
      const int x = warp - 12;            // the warp's tile
      const uint32_t tS = tmem + 128 * x, tO = tmem + 256 + 128 * x, q_tile = base_s + L::Q + x * L::kTile;
      uint32_t c = 0, ns = 0, nq = 0;     // steps, steps of the tile, query tiles
      auto commit = [&](int i) {
        if (elect_one()) tc_commit(bar_at(i));
        __syncwarp();
      };
      while (!fault && wk.next(a, TPT)) {
        const int ja = max(wk.j0, x ? wk.it.a[1] : wk.it.a[0]), je = min(wk.j1, x ? wk.it.e[1] : wk.it.e[0]);
        // Scores against tokens 64 h .. 64 h + 63 of a K stage.
        auto scores = [&](int h, uint32_t cj) {
          if (elect_one())
            mma_scores<D>(tS + 64 * h, smem_desc(q_tile), smem_desc(base_s + L::K + (cj & 1) * L::kTile + h * 64 * 128),
                          bar_at(B_S + 2 * x + h));
          __syncwarp();
        };
        if (!kv8_wait(bar_at(B_KF + (c & 1)), (c >> 1) & 1, a.tries)) { fault = true; break; }
        if (ja < je) {
          if (!kv8_wait(bar_at(B_Q + x), nq++ & 1, a.tries)) { fault = true; break; }
          tc_after_sync();
          if (wk.j0 == ja) {
            scores(0, c);
            scores(1, c);
          }
        }
        commit(B_KE + (c & 1));
        for (int j = wk.j0; j < wk.j1; ++j, ++c) {
          const bool more = j + 1 < wk.j1, here = j >= ja && j < je, there = j + 1 >= ja && j + 1 < je;
          if (!kv8_wait(bar_at(B_VF + (c & 1)), (c >> 1) & 1, a.tries)) { fault = true; break; }
          if (more && !here && !kv8_wait(bar_at(B_KF + ((c + 1) & 1)), ((c + 1) >> 1) & 1, a.tries)) { fault = true; break; }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (here) {
              if (!kv8_wait(bar_at(B_P + 2 * x + h), ns & 1, a.tries)) { fault = true; break; }
              tc_after_sync();
              if (elect_one())
                mma_values<D>(tO, tS + 64 * h, v_desc(base_s + L::V + (c & 1) * L::kTile + h * 64 * 128, L::kHalf),
                              j > ja || h > 0, bar_at(B_O + 2 * x + h));
              __syncwarp();
              if (more && h == 0 && !kv8_wait(bar_at(B_KF + ((c + 1) & 1)), ((c + 1) >> 1) & 1, a.tries)) { fault = true; break; }
            }
            if (there) scores(h, c + 1);
          }
          if (fault) break;
          ns += here;
          commit(B_VE + (c & 1));
          if (more) commit(B_KE + ((c + 1) & 1));
        }
      }
      commit(B_DONE);
      kv8_wait(bar_at(B_DONE), 0, kKv8Tries);
    }
    __syncwarp();
  } else {
    // ---- softmax ------------------------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(PF_REGS_S));
    const int x = warp >> 2, w4 = warp & 3;
    const uint32_t lanes = (uint32_t)(32 * w4) << 16;
    const uint32_t tS = tmem + lanes + 128 * x, tO = tmem + lanes + 256 + 128 * x;
    float* qf = reinterpret_cast<float*>(base + L::QF) + 128 * x;
    const float4* sc = reinterpret_cast<const float4*>(base + L::SC);
    const int row = 32 * w4 + lane;
    const uint32_t invG = 65536u / a.G + 1, q_tile = base_s + L::Q + x * L::kTile;
    const int tok = (int)((row * invG) >> 16);
    uint32_t c = 0, ns = 0;   // steps, steps of the tile
    bool has0 = false, has1 = false;
    // The tile's steps and tokens in the walk's part.
    auto first = [&](const Walk& w) { return max(w.j0, x ? w.it.a[1] : w.it.a[0]); };
    auto last = [&](const Walk& w) { return min(w.j1, x ? w.it.e[1] : w.it.e[0]); };
    auto fetch = [&]() {   // queries of the walk's part
      if (first(wk) < last(wk))
        Queries<D>::copy(a, wk.it.row0 + x * TPT, min(wk.it.ntok - x * TPT, TPT), wk.ih, invG, q_tile, w4, lane);
    };
    auto prepare = [&]() {   // and hand them to the MMA warp
      cp_wait<0>();
      Queries<D>::convert(a, q_tile, qf, w4, lane);
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_at(B_Q + x));
    };
    bool more = wk.next(a, TPT), ready = false;
    if (more) fetch();
    while (more && !fault) {
      const int ja = first(wk), je = last(wk), ntok = min(wk.it.ntok - x * TPT, TPT);
      const int row0 = wk.it.row0 + x * TPT, p_b = wk.ib, p_qt = wk.iqt, p_h = wk.ih, j0 = wk.j0, steps = wk.j1 - wk.j0;
      const bool begun = wk.begun, ended = wk.ended;
      const bool live = tok < ntok && row < TPT * a.G;
      const int pos = wk.it.pos0 + x * TPT + tok;
      const int seen_lo = a.window > 0 ? pos - a.window + 1 : 0, seen_hi = min(pos + 1, wk.it.hi);
      more = wk.next(a, TPT);
      float m = -INFINITY, l = 0.f;
      if (ja >= je && more) fetch();
      if (ja < je) {
        if (!ready) prepare();
        const float f = qf[row];
        // Halves whose tokens every row of the warp sees.
        const int all_lo = __reduce_max_sync(0xffffffffu, live ? seen_lo : 0);
        const int all_hi = __reduce_min_sync(0xffffffffu, live ? seen_hi : 0x7fffffff);
        // Tokens that any of them sees.
        const int any_lo = __reduce_min_sync(0xffffffffu, live ? seen_lo : 0x7fffffff);
        const int any_hi = __reduce_max_sync(0xffffffffu, live ? seen_hi : 0);
        bool begin = true;   // nothing weighed yet
        bool unset = true;   // a row has no reference: no token with a page so far
        const uint32_t bar_s = bar_at(B_S + 2 * x), bar_p = bar_at(B_P + 2 * x);
        // The weights are there: the value product of half h may start.
        auto arrive = [&](int h) {
          tm_wait_st();
          tc_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_p + 8 * h);
        };
        // The common half takes no maximum: the reference stays, and false says
        // that a sum has grown past kMostSum.
        auto weigh = [&](uint32_t tH, const float4* g) {
          uint32_t r[64], p[32];
          tm_ld64(tH, r);
          float most = 0.f, add = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 s4 = g[i];
            const float2 sl = make_float2(f * s4.x, f * s4.x), off = make_float2(s4.y - m, s4.y - m);
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float2 y = fma2(make_float2(__uint_as_float(r[16 * i + 2 * k]), __uint_as_float(r[16 * i + 2 * k + 1])), sl, off);
              y = make_float2(ex2(y.x), ex2(y.y));
              sum = add2(sum, y);
              const __half2 hh = __floats2half2_rn(y.x, y.y);
              p[8 * i + k] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            most = fmaxf(most, sum.x + sum.y);
            add = fmaf(sum.x + sum.y, s4.z, add);
          }
          if (__any_sync(0xffffffffu, most > kMostSum)) return false;
          tm_st32(tH, p);
          l += add;
          return true;
        };
#pragma unroll 1
        for (int jh = 2 * ja; jh < 2 * je; ++jh) {
          const int h = jh & 1, t0 = 64 * jh;
          const uint32_t cj = c + ((jh >> 1) - j0), tH = tS + 64 * h;
          if (!kv8_wait(bar_s + 8 * h, ns & 1, a.tries) || (h == 0 && !kv8_wait(bar_at(B_SC + (cj & 3)), (cj >> 2) & 1, a.tries))) {
            fault = true;
            break;
          }
          tc_after_sync();
          if (more && jh == 2 * je - 1) fetch();   // the last scores are in: the query tile is free
          const float4* g = sc + (cj & 3) * 8 + 4 * h;   // the four groups of 16 tokens
          if (t0 >= any_hi || t0 + 64 <= any_lo) {
            const uint32_t none[32] = {};
            tm_st32(tH, none);
          } else if (unset || t0 < all_lo || t0 + 64 > all_hi || !weigh(tH, g)) {
            // With care: masked tokens, a first or a grown maximum.  (In rolled
            // loops: the roles' code together has to stay in the instruction caches.)
            // Maximum of x_t + log2 w_t over what the row sees.
            float mt = -INFINITY;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t v[16];
              tm_ld16(tH + 16 * i, v);
              const float sl = f * g[i].x, lw = g[i].y;
              const int lo = seen_lo - t0 - 16 * i, hi = seen_hi - t0 - 16 * i;
#pragma unroll
              for (int k = 0; k < 16; ++k)
                if (k >= lo && k < hi) mt = fmaxf(mt, fmaf(__uint_as_float(v[k]), sl, lw));
            }
            // O keeps its reference until a weight passes 2^kLazy.
            const bool grow = mt > m + kLazy;
            if (__any_sync(0xffffffffu, grow)) {
              const float mn = grow ? mt - kBelow : m;
              const float al = m == -INFINITY ? 0.f : ex2(m - mn);
              if (!begin) {
                // O exists: wait for the value product of the half before this
                // one (that half's own scores came after the product before).
                if (!kv8_wait(bar_at(B_O + 2 * x + (h ^ 1)), (ns - (h ^ 1)) & 1, a.tries)) { fault = true; break; }
                tc_after_sync();
                const float fo = m == -INFINITY ? 1.f : al;
#pragma unroll 1
                for (int ch = 0; ch < D / 16; ++ch) {
                  uint32_t o[16];
                  tm_ld16(tO + 16 * ch, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fo);
                  tm_st16(tO + 16 * ch, o);
                }
              }
              l *= al;
              m = mn;
            }
            const float mm = m == -INFINITY ? 0.f : m;
            // Weights, to binary16 over the scores.
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
              uint32_t v[16], p[8];
              tm_ld16(tH + 16 * i, v);
              const float sl = f * g[i].x, off = g[i].y - mm;
              const int lo = seen_lo - t0 - 16 * i, hi = seen_hi - t0 - 16 * i;
              float sum = 0.f;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const float y0 = 2 * k >= lo && 2 * k < hi ? ex2(fmaf(__uint_as_float(v[2 * k]), sl, off)) : 0.f;
                const float y1 = 2 * k + 1 >= lo && 2 * k + 1 < hi ? ex2(fmaf(__uint_as_float(v[2 * k + 1]), sl, off)) : 0.f;
                sum += y0 + y1;
                const __half2 hh = __floats2half2_rn(y0, y1);
                p[k] = *reinterpret_cast<const uint32_t*>(&hh);
              }
              l = fmaf(sum, g[i].z, l);
              tm_st8(tH + 8 * i, p);
            }
            begin = false;
            unset = __any_sync(0xffffffffu, live && m == -INFINITY);
          }
          arrive(h);
          ns += h;
        }
        if (fault) break;
        // The next part's scores run while this one's output is written.
        ready = more && first(wk) < last(wk);
        __syncwarp();   // every lane has its factor
        if (ready) prepare();
        if (!kv8_wait(bar_at(B_O + 2 * x + 1), (ns - 1) & 1, a.tries)) { fault = true; break; }
        tc_after_sync();
      }
      c += steps;
      // ---- output or partial record of the row ---------------------------------------
      const bool whole = begun && ended;
      const int slot = begun ? 1 : 0;
      if (!whole) {
        if (slot) has1 = true; else has0 = true;
        if (tid == 0) {
          JoinHead hd{};
          hd.valid = 1;
          hd.last = ended;
          hd.b = p_b;
          hd.qt = p_qt;
          hd.h = p_h;
          heads[slot] = hd;
        }
        const int64_t rec = ((int64_t)blockIdx.x * 2 + slot) * 256 + 128 * x;
        if (live) reinterpret_cast<float2*>(ws + W.ml)[rec + row] = make_float2(m, l);
        if (ja < je) {
          float* dst = reinterpret_cast<float*>(ws + W.part) + (rec + (row & ~3)) * D + 4 * (lane & 3);
#pragma unroll 1
          for (int ch = 0; ch < D / 16; ++ch) {
            uint32_t r[16];
            tm_ld16(tO + 16 * ch, r);
            uint4 q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) q[i] = make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
            turn4(q, lane);
#pragma unroll
            for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(dst + i * D + 16 * ch) = q[i];   // dead rows too
          }
        }
      } else if (ntok > 0) {
        const float inv = l == 0.f ? 0.f : 1.f / l;   // a row without tokens is 0
        // Of the four rows whose pieces the lane stores: where they go, if they live.
        uint16_t* to[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ri = (row & ~3) + i, ti = (int)((ri * invG) >> 16);
          to[i] = ti < ntok && ri < TPT * a.G ? static_cast<uint16_t*>(a.out) + ((int64_t)(row0 + ti) * a.Hq + (int64_t)p_h * a.G + (ri - ti * a.G)) * D + 8 * (lane & 3)
                                              : nullptr;
        }
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t r[32];
          tm_ld32(tO + 32 * ch, r);
          uint4 q[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t o4[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float u = __uint_as_float(r[8 * i + 2 * k]) * inv, v = __uint_as_float(r[8 * i + 2 * k + 1]) * inv;
              if (a.dtype == TQ_BF16) {
                const __nv_bfloat162 hh = __floats2bfloat162_rn(u, v);
                o4[k] = *reinterpret_cast<const uint32_t*>(&hh);
              } else {
                const __half2 hh = __floats2half2_rn(u, v);
                o4[k] = *reinterpret_cast<const uint32_t*>(&hh);
              }
            }
            q[i] = make_uint4(o4[0], o4[1], o4[2], o4[3]);
          }
          turn4(q, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (to[i]) *reinterpret_cast<uint4*>(to[i] + 32 * ch) = q[i];
        }
      }
      tc_before_sync();
    }
    cp_wait<0>();   // a part that was given up may have queries on their way
    if (tid == 0) {
      if (!has0) heads[0].valid = 0;
      if (!has1) heads[1].valid = 0;
    }
  }
  if (fault) atomicExch(&g_kv8_fault, 1);
  tc_before_sync();
  __syncthreads();
  if (warp == 12) {
    tc_after_sync();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
  }
}

// Joins the parts of an item that several CTAs hold: CTA c that began it
// (record 1), then record 0 of c + 1, ... up to the last.  One warp per row.
template <int D>
__global__ void __launch_bounds__(128) k_kv8_join(Kv8AttnArgs a, int ctas) {
  const int c = blockIdx.x, lane = threadIdx.x & 31, row2 = blockIdx.y * 4 + (threadIdx.x >> 5);
  const char* ws = static_cast<const char*>(a.ws);
  const JoinHead* heads = reinterpret_cast<const JoinHead*>(ws);
  const JoinHead hd = heads[2 * c + 1];
  if (!hd.valid) return;
  const int TPT = PF_TILE / a.G;
  const int x = row2 >> 7, row = row2 & 127, tok = row / a.G, head = row % a.G;
  int row0, count, start;
  ragged_seq(a, hd.b, row0, count, start);
  const int t = hd.qt * 2 * TPT + x * TPT + tok;
  if (row >= TPT * a.G || t >= count) return;
  const PfWs W = pf_ws(D, ctas);
  const float2* ml = reinterpret_cast<const float2*>(ws + W.ml);
  const float* part = reinterpret_cast<const float*>(ws + W.part);
  constexpr int V = D / 32;
  float m = -INFINITY, l = 0.f, o[V];
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = 0.f;
  for (int k = c;; ++k) {
    const int slot = k == c ? 1 : 0;
    const int64_t rec = ((int64_t)k * 2 + slot) * 256 + row2;
    const float2 v = ml[rec];
    if (v.y != 0.f) {   // NaN included; a part without tokens has no O
      const float mn = fmaxf(m, v.x), fo = ex2(m - mn), fn = ex2(v.x - mn);
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = o[i] * fo + fn * part[rec * D + V * lane + i];
      l = l * fo + fn * v.y;
      m = mn;
    }
    if (heads[2 * k + slot].last || k + 1 >= ctas) break;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = ((int64_t)(row0 + t) * a.Hq + (int64_t)hd.h * a.G + head) * D + V * lane;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float u = l == 0.f ? 0.f : o[i] * inv;
    if (a.dtype == TQ_BF16)
      static_cast<__nv_bfloat16*>(a.out)[at + i] = __float2bfloat16_rn(u);
    else
      static_cast<__half*>(a.out)[at + i] = __float2half_rn(u);
  }
}

template <int D>
cudaError_t run_prefill(const Kv8AttnArgs& a, int sms, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_kv8_prefill<D>, PfLayout<D>::total, done);
  if (e != cudaSuccess) return e;
  k_kv8_prefill<D><<<sms, PF_THREADS, PfLayout<D>::total, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  k_kv8_join<D><<<dim3(sms, 64), 128, 0, s>>>(a, sms);
  return cudaGetLastError();
}

size_t decode_part(int B, int d, int sms) { return (kv8_decode_workspace(B, d, sms) + 255) & ~(size_t)255; }

}  // namespace

size_t kv8_prefill_workspace(int B, int d, int sms) {
  return decode_part(B, d, sms) + pf_ws(d, sms).total;
}

// The lengths are on the device, so the host knows the average rows of a
// sequence and not who has them: both kernels run, and each leaves the other's
// sequences out.  The one that finds none costs about 13 us, so one runs alone
// where the other could gain little over whole tables: the decode kernel where
// all rows fill no more than an item, or come to less than kFewTiles of its tiles;
// this one where single rows in all sequences come to less than kMixed steps.
// Single rows and one prompt, and batches of equal sequences (us, alone and both):
//   63 + a prompt of 600, over 8k tokens    594, 321     32 x 32 over 2k   94, 108
//   31 + 1024, over 2k                      132, 113     32 x 64 over 1k   76, 92
//   15 + 2048, over 4k                      200, 192     16 x 256 over 2k  182, 196
//   7 + 1024, over 2k                       75, 83       17 x 4 over 2k    41, 53
cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, int sms, cudaStream_t s) {
  const int64_t cols = a.n * a.G, cap = (int64_t)a.c.max_blocks * a.c.bs;
  const bool few = cols <= kNarrow * (int64_t)a.B;
  const int64_t tiles = (cols + 15) / 16 * a.c.Hkv * (cap / 16), steps = a.B * (int64_t)a.c.Hkv * (cap / PF_TILE + kItemCost);
  if (few && (cols <= 2 * PF_TILE || tiles < kFewTiles)) return launch_kv8_decode(a, sms, s);
  Kv8AttnArgs w = a;
  if (few || steps >= kMixed) {
    Kv8AttnArgs f = a;
    f.most = kNarrow / a.G;
    w.least = f.most + 1;
    w.ws = static_cast<char*>(a.ws) + decode_part(a.B, a.d, sms);
    const cudaError_t e = launch_kv8_decode(f, sms, s);
    if (e != cudaSuccess) return e;
  }
  return a.d == 128 ? run_prefill<128>(w, sms, s) : run_prefill<64>(w, sms, s);
}

cudaError_t read_and_clear_kv8_fault(int* value) {
  cudaError_t e = cudaMemcpyFromSymbol(value, g_kv8_fault, sizeof(int));
  if (e != cudaSuccess) return e;
  const int zero = 0;
  return cudaMemcpyToSymbol(g_kv8_fault, &zero, sizeof(int));
}

}  // namespace tqk
