// 8-bit paged KV cache (e4m3 codes, one fp32 scale per (page, kv head)):
// argument records and device helpers shared by its kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace tqk {

// Raises a kernel's shared-memory limit to `bytes`, once per device: `done`
// holds a bit per device.  (Devices from 64 on set it every time.)
template <typename K>
inline cudaError_t allow_smem(K* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Both attentions weigh a token by 2^(x + log2 w - M), x its score in log2 and
// w its page's value scale, and add the weight / w to the softmax's sum.  A
// page whose scale is below kLeastScale (2^-100, or not a number) has no
// values: it counts in the sum alone, as if its scale were kNoValue.  M then
// rises above what the values need only where such a token's weight is 2^60
// times a value's, and its share of the sum stays in fp32 as long as the other
// scales are below 2^30 (2^-126 is the least weight).
constexpr float kLeastScale = 7.9e-31f;
constexpr float kNoValue = 8.673617379884035e-19f;   // 2^-60

// Token t of sequence b, kv head h: code row (page * Hkv + h) * bs + t % bs,
// scale page * Hkv + h, with page = table[b * max_blocks + t / bs].
struct Kv8Cache {
  uint8_t* kcodes;
  float* kscale;
  uint8_t* vcodes;
  float* vscale;
  const int32_t* table;
  int max_blocks, bs, Hkv;
  int64_t num_blocks;
};

struct Kv8AppendArgs {
  Kv8Cache c;
  const void *q, *k, *v;   // rows [n][heads][d]; q may be null
  void* q_out;
  int64_t ldq, ldk, ldv, ldqo;
  int dtype, B, Hq, d;
  int64_t n;
  const int32_t* cu_q;
  const int32_t* seq_lens;
  const float* rope;       // [cap][rot]: rot / 2 cosines, then rot / 2 sines
  int rot, interleaved;
};

struct Kv8AttnArgs {
  Kv8Cache c;
  const void* q;
  void* out;
  int dtype, B, Hq, G, d, window;
  int64_t n;               // rows (decode: B)
  const int32_t* cu_q;     // null: one row per sequence
  const int32_t* seq_lens;
  int least, most;         // rows of the sequences that the kernel takes
  float scale_log2;        // softmax scale * log2(e)
  int tries;               // of a wait before it gives up
  void* ws;
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}

template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}

// Tries of a wait for an mbarrier, each of which the hardware holds for a while
// (a few hundred ms in all at most).  Main waits take Kv8AttnArgs::tries, which a
// test may cut to 0; waits for what is in flight keep this limit.
constexpr int kKv8Tries = 1 << 22;

__device__ __forceinline__ bool kv8_wait(uint32_t bar, uint32_t parity, int tries) {
  for (int i = 0; i < tries; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// Position of the first of a sequence's `count` rows; far outside the table it
// behaves like one just outside it.
__device__ __forceinline__ int first_pos(const Kv8AttnArgs& a, int b, int count) {
  return (int)max(min((int64_t)a.seq_lens[b] - count, (int64_t)1 << 30), -((int64_t)1 << 30));
}
// Rows of sequence b of a ragged batch; none where it is the other kernel's.
__device__ __forceinline__ void ragged_seq(const Kv8AttnArgs& a, int b, int& row0, int& count, int& start) {
  const int64_t r0 = min((int64_t)max(a.cu_q[b], 0), a.n), r1 = min((int64_t)max(a.cu_q[b + 1], 0), a.n);
  row0 = (int)r0;
  count = (int)max((int64_t)0, r1 - r0);
  start = first_pos(a, b, count);
  if (count < a.least || count > a.most) count = 0;
}

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, cudaStream_t s);
cudaError_t launch_kv8_decode(const Kv8AttnArgs& a, int sms, cudaStream_t s);
size_t kv8_decode_workspace(int B, int d, int sms);
cudaError_t launch_kv8_prefill(const Kv8AttnArgs& a, int sms, cudaStream_t s);
size_t kv8_prefill_workspace(int B, int d, int sms);
cudaError_t read_and_clear_kv8_fault(int* value);
cudaError_t read_and_clear_kv8_decode_fault(int* value);

// Most sequences of a decode call (the prefix of their tile counts is kept in
// shared memory).
constexpr int kKv8MaxSeqs = 2048;

}  // namespace tqk
