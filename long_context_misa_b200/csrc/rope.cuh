// Rotation of one pair, shared by the rotary kernel and the cache write.
#pragma once

#include "common.cuh"

namespace misa {

// amplitude * (cos, sin) of the angle of position p for a phase increment in
// turns / 2^64.  The 64-bit product wraps modulo whole turns, so no range
// reduction is needed and the angle of position 262143 is as exact as that of
// position 1 (an fp32 angle there would be off by 2^18 * 2^-24 = 2^-6
// radians).  Its top 32 bits, rounded, are a signed fraction of a turn, which
// sincospif takes as an fp32 number: up to 2^-26 turns off.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t phase, int p, float amplitude) {
  const uint64_t turns = phase * (uint64_t)(int64_t)p;
  const int f = (int)(uint32_t)((turns + 0x80000000ull) >> 32);
  float sn, cs;
  sincospif((float)f * 0x1p-31f, &sn, &cs);
  return make_float2(cs * amplitude, sn * amplitude);
}

__device__ __forceinline__ float2 rope_pair(float a, float b, float2 cs) {
  return make_float2(fmaf(a, cs.x, -b * cs.y), fmaf(b, cs.x, a * cs.y));
}

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = bf16x2_to_float2(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// The two 8-element chunks that one thread takes of a row whose rotated part
// is [first, first + rot): unit u < rot/16 holds 8 pairs (half layout: the
// chunks of the pairs' two sides; interleaved: 16 consecutive elements), the
// units behind are consecutive chunks of the kept elements.  Needs rot % 16
// == 0, first % 8 == 0 and (d - rot) % 16 == 0, or the last unit holds one
// chunk only (o2 < 0).
__device__ __forceinline__ bool rope_unit(int u, int d, int rot, int first, int interleaved, int &o1, int &o2) {
  if (u < rot / 16) {
    o1 = first + (interleaved ? 16 * u : 8 * u);
    o2 = interleaved ? o1 + 8 : o1 + rot / 2;
    return true;
  }
  const int c = 16 * (u - rot / 16);
  o1 = c < first ? c : c + rot;
  o2 = c + 8 < first ? c + 8 : c + 8 + rot;
  if (o2 >= d) o2 = -1;
  return false;
}

// cos/sin of the 8 pairs of unit u (pairs 8u .. 8u + 7 in both layouts)
__device__ __forceinline__ void rope_unit_cs(const uint64_t *phase, int u, int p, float amplitude, float2 (&cs)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) cs[i] = rope_cos_sin(__ldg(phase + 8 * u + i), p, amplitude);
}

__device__ __forceinline__ void rope_unit_rotate(float (&a)[8], float (&b)[8], const float2 (&cs)[8],
                                                 int interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = rope_pair(a[2 * i], a[2 * i + 1], cs[i]);
      const float2 z = rope_pair(b[2 * i], b[2 * i + 1], cs[4 + i]);
      a[2 * i] = y.x, a[2 * i + 1] = y.y;
      b[2 * i] = z.x, b[2 * i + 1] = z.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = rope_pair(a[i], b[i], cs[i]);
      a[i] = y.x, b[i] = y.y;
    }
  }
}

// Element e of a row, rotated: for rows outside rope_unit's alignment.
__device__ __forceinline__ float rope_element(const uint16_t *row, int e, const uint64_t *phase, int rot, int first,
                                              int interleaved, int p, float amplitude) {
  const float x = bf16_bits_to_float(row[e]);
  const int r = e - first;
  if (r < 0 || r >= rot) return x;
  const int i = interleaved ? r >> 1 : (r < rot / 2 ? r : r - rot / 2);
  const bool second = interleaved ? (r & 1) : r >= rot / 2;
  const int step = interleaved ? 1 : rot / 2;
  const float2 cs = rope_cos_sin(__ldg(phase + i), p, amplitude);
  const float other = bf16_bits_to_float(row[second ? e - step : e + step]);
  return second ? rope_pair(other, x, cs).y : rope_pair(x, other, cs).x;
}

}  // namespace misa
