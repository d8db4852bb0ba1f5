// Host-side launchers and device views of the attention side
// (misa_attention.h), shared between its translation units.
#pragma once

#include "common.cuh"
#include "misa_attention.h"

namespace misa {

// Device view of the caller's attention cache (by value).
struct KvView {
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  int32_t *seq_len;
  uint32_t *status;
  int n_seq, L_cap, H_kv, d, fp8;
};

__device__ __forceinline__ void flag(const KvView &c, uint32_t bit) {
  if (c.status) atomicOr(c.status, bit);
}

// Two fp32 values in one register pair: sm_100's paired arithmetic.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(a), "f"(b));
  return p;
}
__device__ __forceinline__ float2 unpair(uint64_t p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Rotary parameters of a launch.
struct RopeView {
  const uint64_t *phase;  // nullptr: no rotation
  int rot, first, interleaved;
  float amplitude;
};

// Whether two arrays of int32 share memory.
inline bool overlap(const int32_t *a, int64_t na, const int32_t *b, int64_t nb) { return a < b + nb && b < a + na; }

// Heads that one thread of the rotary and cache kernels takes: `flat` threads
// would take one each.  A thread's 8 cos and sin cost about 350 instructions,
// as many as the memory leaves room for per 64 bytes, so a large call shares
// them over up to 8 heads while half the device's threads remain busy.
inline int heads_per_thread(int64_t flat, int heads) {
  int per = 1;
  while (per < 8 && 2 * per <= heads && flat / (2 * per) >= (int64_t)device_sms() * 1024) per *= 2;
  return per;
}

// rope.cu
cudaError_t launch_rope(const RopeView &r, const misa_rope_rows *groups, int n_groups, cudaStream_t s);

// kvcache.cu
cudaError_t launch_append_kv(const KvView &c, const misa_new_kv &in, const int32_t *new_pos, int count,
                             const RopeView &r, const int32_t *rope_pos, bool commit, cudaStream_t s);
cudaError_t launch_read_kv(const KvView &c, const int32_t *seq, const int32_t *tok, int n, int k, uint16_t *k_out,
                           uint16_t *v_out, cudaStream_t s);

// attend.cu
struct AttendView {
  const uint16_t *q;
  const int32_t *q_seq, *q_pos;
  int n_q, H;
  float scale;
  const int32_t *topk;  // nullptr: whole prefixes
  int k;
  const int32_t *draft_start;  // nullptr: no drafted tokens
  const uint32_t *draft_mask;
  int n_draft;
  uint16_t *out;
  float *lse;
};
size_t attend_ws_bytes(const KvView &c, int n_q, int H, int k, int n_draft);
cudaError_t launch_attend(const KvView &c, const AttendView &a, void *ws, cudaStream_t s);

}  // namespace misa
