// The attention cache: written as tokens arrive (misa_append_kv) and read back
// at listed tokens (misa_read_kv).
//
// Both are bound by their traffic: rows in, rows out, once each.  A row of d
// elements belongs to d/16 neighbouring threads of 16 elements (two 16-byte
// chunks of bf16).
//
// Write, e4m3: scale = amax / 448 (1 for a zero row), code = e4m3(x / scale)
// rounded to nearest even and saturated, in fp32 with IEEE division: the rule
// of misa_append_keys_e4m3.  The key is rotated in fp32 first and not rounded
// in between.  A thread keeps its 8 pairs' cos and sin for the heads of a
// token that it takes one after the other.
#include "attention.h"
#include "frag.cuh"
#include "rope.cuh"

namespace misa {
namespace {

constexpr int THREADS = 256;

// 16 elements (chunks at o1 and o2 of a row) to the cache.  LPR threads hold
// the row; all 32 lanes call.
template <int LPR>
__device__ __forceinline__ void store_row(const float (&a)[8], const float (&b)[8], uint8_t *row, float *scale, int o1,
                                          int o2, bool fp8, bool store, int part) {
  if (!fp8) {
    if (!store) return;
    *reinterpret_cast<uint4 *>(row + 2 * o1) = pack8(a);
    *reinterpret_cast<uint4 *>(row + 2 * o2) = pack8(b);
    return;
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!store) return;
  const float sc = m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = f32x2_to_e4m3x2(__fdiv_rn(a[2 * i], sc), __fdiv_rn(a[2 * i + 1], sc)) & 0xFFFFu;
    c[4 + i] = f32x2_to_e4m3x2(__fdiv_rn(b[2 * i], sc), __fdiv_rn(b[2 * i + 1], sc)) & 0xFFFFu;
  }
  *reinterpret_cast<uint2 *>(row + o1) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  *reinterpret_cast<uint2 *>(row + o2) = make_uint2(c[4] | (c[5] << 16), c[6] | (c[7] << 16));
  if (part == 0) *scale = sc;
}

// LPR = d / 16 threads per row.  VEC: the rotated part fits rope_unit's
// alignment (or nothing is rotated).
template <int LPR, bool VEC>
__global__ void __launch_bounds__(THREADS) append_kv_kernel(KvView c, misa_new_kv in, const int32_t *new_pos,
                                                            int count, RopeView r, const int32_t *rope_pos,
                                                            int commit, int head_groups) {
  grid_dep_sync();
  constexpr int DH = LPR * 16;
  const int64_t t = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  const int part = (int)(t % LPR);
  int64_t rest = t / LPR;
  const int hg = (int)(rest % head_groups);
  rest /= head_groups;
  const int j = (int)(rest % count);
  const int64_t s64 = rest / count;
  const int s = (int)min(s64, (int64_t)c.n_seq - 1);
  bool live = s64 < c.n_seq;
  const int pos = new_pos[s];
  if (pos < 0) live = false;
  if (live && (int64_t)pos + count > c.L_cap) {
    if (part == 0 && hg == 0 && j == 0) flag(c, MISA_DEV_APPEND_RANGE);
    live = false;
  }
  if (live && commit && part == 0 && hg == 0 && j == 0) c.seq_len[s] = pos + count;
  int o1 = 16 * part, o2 = o1 + 8;
  bool rotated = false;
  float2 cs[8];
  int p = 0;
  if (r.phase) {
    p = rope_pos ? rope_pos[(int64_t)s * count + j] : pos + j;
    if (VEC) {
      rotated = rope_unit(part, DH, r.rot, r.first, r.interleaved, o1, o2);
      if (rotated) rope_unit_cs(r.phase, part, p, r.amplitude, cs);
    }
  }
  const uint16_t *k = in.k + s * in.k_seq + j * in.k_tok;
  const uint16_t *v = in.v + s * in.v_seq + j * in.v_tok;
  const int esz = c.fp8 ? 1 : 2;
  const int64_t row0 = ((int64_t)s * c.L_cap + (live ? pos + j : 0)) * c.H_kv;
  // every lane takes every step: a row's amax is reduced over its lanes
  for (int h0 = 0; h0 < c.H_kv; h0 += head_groups) {
    const int h = h0 + hg;
    const bool store = live && h < c.H_kv;
    const int hr = store ? h : 0;
    float a[8], b[8];
    if (VEC) {
      unpack8(*reinterpret_cast<const uint4 *>(k + hr * in.k_head + o1), a);
      unpack8(*reinterpret_cast<const uint4 *>(k + hr * in.k_head + o2), b);
      if (rotated) rope_unit_rotate(a, b, cs, r.interleaved);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] = rope_element(k + hr * in.k_head, o1 + e, r.phase, r.rot, r.first, r.interleaved, p, r.amplitude);
        b[e] = rope_element(k + hr * in.k_head, o2 + e, r.phase, r.rot, r.first, r.interleaved, p, r.amplitude);
      }
    }
    float va[8], vb[8];
    unpack8(*reinterpret_cast<const uint4 *>(v + hr * in.v_head + o1), va);
    unpack8(*reinterpret_cast<const uint4 *>(v + hr * in.v_head + o2), vb);
    const int64_t row = row0 + hr;
    store_row<LPR>(a, b, c.k + row * DH * esz, c.k_scale + (c.fp8 ? row : 0), o1, o2, c.fp8, store, part);
    store_row<LPR>(va, vb, c.v + row * DH * esz, c.v_scale + (c.fp8 ? row : 0), o1, o2, c.fp8, store, part);
  }
}

// Thread: 16 elements of one row of the keys or (second half of the grid's y)
// the values.
template <int LPR>
__global__ void __launch_bounds__(THREADS) read_kv_kernel(KvView c, const int32_t *seq, const int32_t *tok,
                                                          int64_t rows, int k, uint16_t *k_out, uint16_t *v_out) {
  grid_dep_sync();
  constexpr int DH = LPR * 16;
  const bool keys = k_out && blockIdx.y == 0;
  uint16_t *out = keys ? k_out : v_out;
  const uint8_t *src = keys ? c.k : c.v;
  const float *scale = keys ? c.k_scale : c.v_scale;
  const int64_t t = (int64_t)blockIdx.x * THREADS + threadIdx.x;
  const int part = (int)(t % LPR);
  const int64_t orow = t / LPR;  // (i * k + j) * H_kv + h
  if (orow >= rows) return;
  const int64_t ij = orow / c.H_kv;
  const int h = (int)(orow - ij * c.H_kv);
  const int s = seq[ij / k], token = tok[ij];
  uint4 *dst = reinterpret_cast<uint4 *>(out + orow * DH) + 2 * part;
  const bool there = s >= 0 && s < c.n_seq && token >= 0 && token < c.L_cap;
  if (!there) {
    if (token != -1 || s < 0 || s >= c.n_seq) flag(c, MISA_DEV_BAD_POSITION);
    dst[0] = dst[1] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const int64_t row = ((int64_t)s * c.L_cap + token) * c.H_kv + h;
  if (!c.fp8) {
    const uint4 *p = reinterpret_cast<const uint4 *>(src + row * DH * 2) + 2 * part;
    const uint4 a = p[0], b = p[1];
    dst[0] = a;
    dst[1] = b;
    return;
  }
  const uint4 w = *(reinterpret_cast<const uint4 *>(src + row * DH) + part);
  const float sc = scale[row];
  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 lo = e4m3x2_to_f32x2(ww[i] & 0xFFFFu), hi = e4m3x2_to_f32x2(ww[i] >> 16);
    o[2 * i] = pack_bf16(lo.x * sc, lo.y * sc);
    o[2 * i + 1] = pack_bf16(hi.x * sc, hi.y * sc);
  }
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

}  // namespace

cudaError_t launch_append_kv(const KvView &c, const misa_new_kv &in, const int32_t *new_pos, int count,
                             const RopeView &r, const int32_t *rope_pos, bool commit, cudaStream_t s) {
  const int lpr = c.d / 16;
  // heads per thread as in the rotary kernel: several only where the threads
  // fill the device twice over
  const int64_t flat = (int64_t)c.n_seq * count * c.H_kv * lpr, full = (int64_t)device_sms() * 4096;
  int per = 1;
  while (per < 8 && per < c.H_kv && flat / (2 * per) >= full) per *= 2;
  const int head_groups = cdiv(c.H_kv, per);
  const int64_t blocks = ((int64_t)c.n_seq * count * head_groups * lpr + THREADS - 1) / THREADS;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const bool vec = !r.phase || (r.rot % 16 == 0 && r.first % 8 == 0);
  const dim3 g((unsigned)blocks), b(THREADS);
  const int cm = commit ? 1 : 0;
  if (c.d == 128)
    return vec ? launch_kernel(append_kv_kernel<8, true>, g, b, 0, s, c, in, new_pos, count, r, rope_pos, cm, head_groups)
               : launch_kernel(append_kv_kernel<8, false>, g, b, 0, s, c, in, new_pos, count, r, rope_pos, cm, head_groups);
  return vec ? launch_kernel(append_kv_kernel<4, true>, g, b, 0, s, c, in, new_pos, count, r, rope_pos, cm, head_groups)
             : launch_kernel(append_kv_kernel<4, false>, g, b, 0, s, c, in, new_pos, count, r, rope_pos, cm, head_groups);
}

cudaError_t launch_read_kv(const KvView &c, const int32_t *seq, const int32_t *tok, int n, int k, uint16_t *k_out,
                           uint16_t *v_out, cudaStream_t s) {
  const int64_t rows = (int64_t)n * k * c.H_kv;
  if (rows == 0) return cudaSuccess;
  const int64_t blocks = (rows * (c.d / 16) + THREADS - 1) / THREADS;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  const dim3 g((unsigned)blocks, k_out && v_out ? 2 : 1), b(THREADS);
  return c.d == 128 ? launch_kernel(read_kv_kernel<8>, g, b, 0, s, c, seq, tok, rows, k, k_out, v_out)
                    : launch_kernel(read_kv_kernel<4>, g, b, 0, s, c, seq, tok, rows, k, k_out, v_out);
}

}  // namespace misa
