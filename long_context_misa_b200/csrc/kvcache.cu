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
//
// Measured, 8 key/value heads of 128, a call in a row of them / alone in a graph.
// Write of 2 x 8192 rotated tokens to e4m3 (102 MB): 24.2 us, 4.2 TB/s / 26.6 (28.7
// with codes taken at both ends of an interval around the quotient and an fp64
// product where they differed).  Read of 8 x 2048 listed e4m3 tokens (102 MB with
// the outputs): 19.1 us, 5.3 TB/s / 20.7; forms with fewer instructions (row
// numbers by multiplication, paired products) and with two pieces per thread took
// 21.2 to 22.6 alone.  A few rows: 2.4 / 4.1 us either way, the launch and its
// dependent loads.
#include <algorithm>

#include "attention.h"
#include "frag.cuh"
#include "rope.cuh"

namespace misa {
namespace {

constexpr int THREADS = 128;

// Two e4m3 codes (nearest even, saturated), a's in the low byte.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(c) : "f"(a), "f"(b));
  return c;
}

// e4m3(f / sc) of 8 elements, f / sc rounded to fp32 in between.
// near: y = 1 / sc rounded.  One correction of the product (P. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor",
// IBM J. Res. Dev. 34, 1990): q0 = f y, q = q0 + y (f - sc q0).  q0 is within 2
// ulp of f / sc, 1 - sc y within 2^-24, the remainder's rounding adds 2^-24 ulp:
// before its last rounding q is within 3 * 2^-24 ulp of f / sc.  The code of q can
// differ from that of the rounded quotient only where f / sc lies that close
// to M + half an ulp or M - half an ulp, M a boundary between codes.  In half
// ulps, with f = A 2^i, sc = B 2^j (A, B of 24 bits) and M = m 2^20 (m of 5
// bits), that is |A 2^k - B (m 2^20 +- 1)| <= 6 * 2^-24 B < 6, k >= 24: a
// nonzero B modulo 2^20 within 6 of 0.  near excludes such B; B = 0 modulo 2^20
// leaves no number but 0 there, and 0 rounds alike.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float sc, float y, bool near) {
  float q[8];
  if (near) {
    // (-q is computed: that way around a -0 stays one)
    const uint64_t yy = pair(-y, -y), ss = pair(sc, sc);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const uint64_t x = pair(f[i], f[i + 1]), q0 = mul2(x, yy);
      const float2 t = unpair(fma2(fma2(ss, q0, x), yy, q0));
      q[i] = -t.x, q[i + 1] = -t.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(f[i], sc);
  }
  return make_uint2(codes2(q[0], q[1]) | codes2(q[2], q[3]) << 16, codes2(q[4], q[5]) | codes2(q[6], q[7]) << 16);
}

// 16 elements (chunks at o1 and o2 of a row) to the cache.  LPR threads hold
// the row; all 32 lanes call.
template <int LPR, bool FP8>
__device__ __forceinline__ void store_row(const float (&a)[8], const float (&b)[8], uint8_t *cache, float *scales,
                                          int64_t row, int o1, int o2, bool store, int part) {
  if (!FP8) {
    if (!store) return;
    uint16_t *to = reinterpret_cast<uint16_t *>(cache) + row * (LPR * 16);
    *reinterpret_cast<uint4 *>(to + o1) = pack8(a);
    *reinterpret_cast<uint4 *>(to + o2) = pack8(b);
    return;
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fmaxf(fabsf(a[i]), fabsf(b[i])));
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (!store) return;
  // m / 448, corrected once as in codes8: the divisor's significand is 7 * 2^21,
  // so no quotient lies nearer to a midpoint than a seventh of half an ulp
  constexpr float R448 = 1.f / 448.f;
  const float s0 = m * R448;
  const bool normal = m >= 0x1p-71f && m <= 0x1p120f;  // no remainder below fp32's range, nothing infinite
  const float sc = normal ? fmaf(fmaf(-448.f, s0, m), R448, s0) : m > 0.f ? __fdiv_rn(m, 448.f) : 1.f;
  const uint32_t low = __float_as_uint(sc) & 0xFFFFFu;
  const bool near = (normal || m == 0.f) && (low == 0u || (low > 7u && low < 0x100000u - 7u));
  const float inv = __frcp_rn(sc);
  const uint2 x = codes8(a, sc, inv, near), y = codes8(b, sc, inv, near);
  uint8_t *to = cache + row * (LPR * 16);
  if (o2 == o1 + 8 && (o1 & 15) == 0) {
    *reinterpret_cast<uint4 *>(to + o1) = make_uint4(x.x, x.y, y.x, y.y);
  } else {
    *reinterpret_cast<uint2 *>(to + o1) = x;
    *reinterpret_cast<uint2 *>(to + o2) = y;
  }
  if (part == 0) scales[row] = sc;
}

// LPR = d / 16 threads per row.  ROT: nothing is rotated, or a part that fits
// rope_unit's alignment, or any part.
constexpr int ROT_NONE = 0, ROT_VEC = 1, ROT_ANY = 2;

template <int LPR, bool FP8, int ROT>
__global__ void __launch_bounds__(THREADS, 5) append_kv_kernel(KvView c, misa_new_kv in, const int32_t *new_pos,
                                                            int count, RopeView r, const int32_t *rope_pos,
                                                            int commit, int head_groups) {
  grid_dep_sync();
  constexpr int DH = LPR * 16;
  // blockIdx.x: the (token, head group, part)s of a sequence, below 2^28
  const uint32_t t = blockIdx.x * THREADS + threadIdx.x, rest = t / LPR;
  const int part = (int)(t % LPR), j0 = (int)(rest / (uint32_t)head_groups);
  const int hg = (int)(rest - (uint32_t)j0 * head_groups), j = min(j0, count - 1);
  for (int s = blockIdx.y; s < c.n_seq; s += gridDim.y) {
    bool live = j0 < count;
    const int pos = new_pos[s];
    if (pos < 0) live = false;
    if (live && (int64_t)pos + count > c.L_cap) {
      if (part == 0 && hg == 0 && j == 0) flag(c, MISA_DEV_APPEND_RANGE);
      live = false;
    }
    if (live && commit && part == 0 && hg == 0 && j == 0) c.seq_len[s] = pos + count;
    int o1 = 16 * part, o2 = o1 + 8;
    const bool rotated = ROT == ROT_VEC && rope_unit(part, DH, r.rot, r.first, r.interleaved, o1, o2);
    const uint16_t *k = in.k + s * in.k_seq + j * in.k_tok;
    const uint16_t *v = in.v + s * in.v_seq + j * in.v_tok;
    uint4 raw[4];  // a head's key and value chunks, read one head ahead
    auto read = [&](int h) {
      const int hr = h < c.H_kv ? h : 0;
      if (ROT != ROT_ANY) {
        raw[0] = *reinterpret_cast<const uint4 *>(k + hr * in.k_head + o1);
        raw[1] = *reinterpret_cast<const uint4 *>(k + hr * in.k_head + o2);
      }
      raw[2] = *reinterpret_cast<const uint4 *>(v + hr * in.v_head + o1);
      raw[3] = *reinterpret_cast<const uint4 *>(v + hr * in.v_head + o2);
    };
    read(hg);
    float2 cs[8];
    int p = 0;
    if (ROT != ROT_NONE) p = rope_pos ? rope_pos[(int64_t)s * count + j] : pos + j;
    if (rotated) rope_unit_cs(r.phase, part, p, r.amplitude, cs);
    const int64_t row0 = ((int64_t)s * c.L_cap + (live ? pos + j : 0)) * c.H_kv;
    // every lane takes every step: a row's amax is reduced over its lanes
    for (int h0 = 0; h0 < c.H_kv; h0 += head_groups) {
      const int h = h0 + hg;
      const bool store = live && h < c.H_kv;
      const int hr = store ? h : 0;
      float a[8], b[8], va[8], vb[8];
      if (ROT != ROT_ANY) {
        unpack8(raw[0], a);
        unpack8(raw[1], b);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] = rope_element(k + hr * in.k_head, o1 + e, r.phase, r.rot, r.first, r.interleaved, p, r.amplitude);
          b[e] = rope_element(k + hr * in.k_head, o2 + e, r.phase, r.rot, r.first, r.interleaved, p, r.amplitude);
        }
      }
      unpack8(raw[2], va);
      unpack8(raw[3], vb);
      if (h0 + head_groups < c.H_kv) read(h + head_groups);
      if (rotated) rope_unit_rotate(a, b, cs, r.interleaved);
      const int64_t row = row0 + hr;
      store_row<LPR, FP8>(a, b, c.k, c.k_scale, row, o1, o2, store, part);
      store_row<LPR, FP8>(va, vb, c.v, c.v_scale, row, o1, o2, store, part);
    }
  }
}

// seq_len where the cache's own lengths said where the tokens go: the write
// reads them, so they change once it is done.
__global__ void commit_kv_kernel(KvView c, const int32_t *new_pos, int count) {
  grid_dep_sync();
  const int s = blockIdx.x * THREADS + threadIdx.x;
  if (s >= c.n_seq) return;
  const int pos = new_pos[s];
  if (pos >= 0 && (int64_t)pos + count <= c.L_cap) c.seq_len[s] = pos + count;
}

// blockIdx.z: keys or values; blockIdx.y: list; blockIdx.x: the list's
// pieces of 8 elements, READ_PIECES of them per thread, THREADS apart: a warp
// stores 512 contiguous bytes at a time.
constexpr int READ_PIECES = 4;

template <int DH>
__global__ void __launch_bounds__(THREADS) read_kv_kernel(KvView c, const int32_t *seq, const int32_t *tok, int n,
                                                          int k, uint16_t *k_out, uint16_t *v_out) {
  grid_dep_sync();
  constexpr uint32_t PPR = DH / 8;  // pieces per row
  const bool keys = k_out && blockIdx.z == 0;
  uint16_t *out = keys ? k_out : v_out;
  const uint8_t *src = keys ? c.k : c.v;
  const float *scale = keys ? c.k_scale : c.v_scale;
  const uint32_t total = (uint32_t)k * c.H_kv * PPR;  // at most 2^29
  for (int i = blockIdx.y; i < n; i += gridDim.y) {
    const int s = seq[i];
    const bool seq_ok = s >= 0 && s < c.n_seq;
    uint4 v[READ_PIECES];
    float sc[READ_PIECES];
#pragma unroll
    for (int u = 0; u < READ_PIECES; ++u) {
      const uint32_t e = blockIdx.x * (THREADS * READ_PIECES) + u * THREADS + threadIdx.x;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      sc[u] = 1.f;
      if (e >= total) continue;
      const uint32_t row = e / PPR, j = row / (uint32_t)c.H_kv;
      const int token = tok[(int64_t)i * k + j];
      if (!seq_ok || token < 0 || token >= c.L_cap) {
        if (token != -1 || !seq_ok) flag(c, MISA_DEV_BAD_POSITION);
        continue;
      }
      const int64_t at = ((int64_t)s * c.L_cap + token) * c.H_kv + (row - j * c.H_kv);
      if (c.fp8) {
        const uint2 w = *reinterpret_cast<const uint2 *>(src + at * DH + (e % PPR) * 8);
        v[u].x = w.x, v[u].y = w.y;
        sc[u] = scale[at];
      } else {
        v[u] = *reinterpret_cast<const uint4 *>(src + at * DH * 2 + (e % PPR) * 16);
      }
    }
#pragma unroll
    for (int u = 0; u < READ_PIECES; ++u) {
      const uint32_t e = blockIdx.x * (THREADS * READ_PIECES) + u * THREADS + threadIdx.x;
      if (e >= total) continue;
      uint4 o = v[u];
      if (c.fp8) {
        const float2 a = e4m3x2_to_f32x2(v[u].x & 0xFFFFu), b = e4m3x2_to_f32x2(v[u].x >> 16);
        const float2 d = e4m3x2_to_f32x2(v[u].y & 0xFFFFu), f = e4m3x2_to_f32x2(v[u].y >> 16);
        o = make_uint4(pack_bf16(a.x * sc[u], a.y * sc[u]), pack_bf16(b.x * sc[u], b.y * sc[u]),
                       pack_bf16(d.x * sc[u], d.y * sc[u]), pack_bf16(f.x * sc[u], f.y * sc[u]));
      }
      *reinterpret_cast<uint4 *>(out + ((int64_t)i * total + e) * 8) = o;
    }
  }
}

}  // namespace

cudaError_t launch_append_kv(const KvView &c, const misa_new_kv &in, const int32_t *new_pos, int count,
                             const RopeView &r, const int32_t *rope_pos, bool commit, cudaStream_t s) {
  const int lpr = c.d / 16;
  const bool after = commit && (overlap(new_pos, c.n_seq, c.seq_len, c.n_seq) ||
                                (rope_pos && overlap(rope_pos, (int64_t)c.n_seq * count, c.seq_len, c.n_seq)));
  // without a rotation there is nothing to share between heads
  const int per = heads_per_thread((int64_t)c.n_seq * count * c.H_kv * lpr, r.phase ? c.H_kv : 1);
  const int head_groups = cdiv(c.H_kv, per);
  const int blocks = cdiv(count * head_groups * lpr, THREADS);  // below 2^28 threads
  const int rot = !r.phase ? ROT_NONE : r.rot % 16 == 0 && r.first % 8 == 0 ? ROT_VEC : ROT_ANY;
  const dim3 g((unsigned)blocks, (unsigned)std::min(c.n_seq, 65535)), b(THREADS);
  auto go = [&](auto kernel) {
    return launch_kernel(kernel, g, b, 0, s, c, in, new_pos, count, r, rope_pos, commit && !after ? 1 : 0,
                         head_groups);
  };
  auto by_rot = [&](auto none, auto vec, auto any) {
    return rot == ROT_NONE ? go(none) : rot == ROT_VEC ? go(vec) : go(any);
  };
  cudaError_t e;
  if (c.d == 128)
    e = c.fp8 ? by_rot(append_kv_kernel<8, true, ROT_NONE>, append_kv_kernel<8, true, ROT_VEC>,
                       append_kv_kernel<8, true, ROT_ANY>)
              : by_rot(append_kv_kernel<8, false, ROT_NONE>, append_kv_kernel<8, false, ROT_VEC>,
                       append_kv_kernel<8, false, ROT_ANY>);
  else
    e = c.fp8 ? by_rot(append_kv_kernel<4, true, ROT_NONE>, append_kv_kernel<4, true, ROT_VEC>,
                       append_kv_kernel<4, true, ROT_ANY>)
              : by_rot(append_kv_kernel<4, false, ROT_NONE>, append_kv_kernel<4, false, ROT_VEC>,
                       append_kv_kernel<4, false, ROT_ANY>);
  if (e != cudaSuccess || !after) return e;
  return launch_kernel(commit_kv_kernel, dim3((unsigned)cdiv(c.n_seq, THREADS)), b, 0, s, c, new_pos, count);
}

cudaError_t launch_read_kv(const KvView &c, const int32_t *seq, const int32_t *tok, int n, int k, uint16_t *k_out,
                           uint16_t *v_out, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const int blocks = cdiv(k * c.H_kv * (c.d / 8), THREADS * READ_PIECES);  // at most 2^29 pieces
  const dim3 g((unsigned)blocks, (unsigned)std::min(n, 65535), k_out && v_out ? 2 : 1), b(THREADS);
  return c.d == 128 ? launch_kernel(read_kv_kernel<128>, g, b, 0, s, c, seq, tok, n, k, k_out, v_out)
                    : launch_kernel(read_kv_kernel<64>, g, b, 0, s, c, seq, tok, n, k, k_out, v_out);
}

}  // namespace misa
