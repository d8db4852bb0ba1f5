// What the attention kernels share: numeric helpers, the tiles of a batch of
// queries, and the join of a row's parts.
#pragma once

#include "attention.h"

namespace misa {

// Binary orders between a row's largest weight and its reference when that
// moves, and most that a weight may reach before it does.  e4m3 caches: f16
// holds weights from 2^-25 to 2^16, so the largest starts at 2^7 and what is
// lost lies 2^-32 below it (2^18 tokens of it: 2^-14); 2^8 times as much may
// come without a move, as with bf16, whose range is fp32's.
template <bool FP8>
constexpr float BELOW = FP8 ? 7.f : 0.f;
template <bool FP8>
constexpr float LAZY = FP8 ? 0x1p15f : 256.f;
// most that a chunk's weights may add to a row's sum before the reference moves:
// rows of scale 0 add nothing to O, whatever they weigh (2^18 tokens of such
// chunks still fit fp32)
constexpr float SUM_MAX = 0x1p110f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float NEG_INF = -__builtin_huge_valf();
// reference of a row that has seen nothing: finite, so that a logit of -inf
// still weighs 0 against it, and far enough down that any other logit moves it
constexpr float NOTHING = -3e38f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Four e4m3 codes -> their exact f16 values, two to a register.
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// 2^(7 - E) for amax = m 2^E, m in [0.5, 1): the largest element lands in
// [64, 128).  1 for zeros.
__device__ __forceinline__ float f16_scale(float amax) {
  if (!(amax > 0.f)) return 1.f;
  const int e = 7 - ((int)(__float_as_uint(amax) >> 23) - 126);
  return __uint_as_float((uint32_t)(min(max(e, -126), 126) + 127) << 23);
}
// 1 / s of such a power of two, by its exponent
__device__ __forceinline__ float inverse(float s) { return __uint_as_float(0x7f000000u - __float_as_uint(s)); }

// max(m, |x|), where x is finite
__device__ __forceinline__ float finite_max(float m, float x) {
  const float y = fabsf(x);
  return y < __int_as_float(0x7f800000) ? fmaxf(m, y) : m;
}

// log2 of a value scale for the reference of O, held within [-93, 100]: a row
// of zeros (scale 0) or one that held an infinity must not move the others'
// reference out of fp32's range.
__device__ __forceinline__ float log2_scale(float s) { return __log2f(fminf(fmaxf(s, 0x1p-93f), 0x1p100f)); }

// The reference that a visible token of logit x and value scale vs asks for.
// From 2^24 on an fp32 reference has no room for more than the logit: the
// scale's power of two, rounded away or up, could cost or overflow the weight.
template <bool FP8>
__device__ __forceinline__ float reference(float x, float vs) {
  if (!FP8) return x;
  const float y = x + (log2_scale(vs) - BELOW<true>);
  return fabsf(x) < 0x1p24f ? y : x;
}

// Prefix length of query i (0 for none) and its sequence (-1: outside the
// cache, it sees nothing).
__device__ __forceinline__ int attend_prefix(const KvView &c, const AttendView &a, int i, int *seq) {
  const int s = a.q_seq[i], p = a.q_pos[i];
  if (s < 0 || s >= c.n_seq || p < -1) {
    flag(c, MISA_DEV_BAD_POSITION);
    *seq = -1;
    return 0;
  }
  *seq = s;
  const int len = max(min(c.seq_len[s], c.L_cap), 0);
  if (p >= len) {
    flag(c, MISA_DEV_BAD_POSITION);
    return len;
  }
  return p + 1;
}

// Queries [q0, q0 + n) of one sequence that a tile holds, and the batch's
// number of tiles.
struct Tile {
  int q0, n, total;
};

// Tile number `want` of the batch without lists: runs of neighbouring queries
// of one sequence (cut at multiples of 1024 queries) are dealt to tiles of up
// to `per` queries, in order.  Every thread of the block calls, the first
// THREADS of them look; n == 0 when there is no such tile.
template <int THREADS>
__device__ Tile find_tile(const AttendView &a, int per, int want) {
  constexpr int SPAN = 1024, PER_T = SPAN / THREADS, NWARP = THREADS / 32;
  __shared__ int seq_s[SPAN];
  __shared__ int part[NWARP + 1];
  __shared__ Tile found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) found = {0, 0, 0};
  int tiles = 0;
  for (int base = 0; base < a.n_q; base += SPAN) {
    const int m = min(SPAN, a.n_q - base);
    __syncthreads();
    for (int i = tid; i < m; i += blockDim.x) seq_s[i] = a.q_seq[base + i];
    __syncthreads();
    // start of each query's run: a running maximum of the run starts
    int start[PER_T], mx = 0;
#pragma unroll
    for (int e = 0; e < PER_T; ++e) {
      const int i = tid * PER_T + e;
      if (i < m && i > 0 && seq_s[i] != seq_s[i - 1]) mx = i;
      start[e] = mx;
    }
    int incl = mx;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = max(incl, x);
    }
    int before = __shfl_up_sync(0xffffffffu, incl, 1);
    if (lane == 0) before = 0;
    if (lane == 31 && warp < NWARP) part[warp] = incl;
    __syncthreads();
    for (int w = 0; w < min(warp, NWARP); ++w) before = max(before, part[w]);
    // queries that lead a tile, counted in order
    int lead = 0;
    bool is[PER_T];
#pragma unroll
    for (int e = 0; e < PER_T; ++e) {
      const int i = tid * PER_T + e;
      is[e] = i < m && (i - max(start[e], before)) % per == 0;
      lead += is[e];
    }
    int sum = lead;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    __syncthreads();
    if (lane == 31 && warp < NWARP) part[warp] = sum;
    __syncthreads();
    int first = sum - lead, total = 0;
    for (int w = 0; w < NWARP; ++w) {
      if (w < warp) first += part[w];
      total += part[w];
    }
#pragma unroll
    for (int e = 0; e < PER_T; ++e) {
      if (!is[e]) continue;
      if (tiles + first++ == want) {
        const int i = tid * PER_T + e;
        int n = 1;
        while (n < per && i + n < m && seq_s[i + n] == seq_s[i]) ++n;
        found = {base + i, n, 0};
      }
    }
    tiles += total;
  }
  __syncthreads();
  Tile t = found;
  t.total = tiles;
  __syncthreads();
  return t;
}

struct Split {
  float *o;    // [Z][n_q * H][DH]; nullptr: the Z shares are a cluster
  float2 *yl;  // [Z][n_q * H] (reference, sum)
  int Z;
};

// A part of a row: O and the sum of weights, both relative to 2^Y.
struct Part {
  float Y = NOTHING, l = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
};

// Join n parts: yl(i) = (reference, sum), v(i) = 4 elements of O.
template <int UNROLL, class YL, class V>
__device__ __forceinline__ Part join_parts(int n, YL &&yl, V &&v) {
  Part p;
#pragma unroll UNROLL
  for (int i = 0; i < n; ++i) p.Y = fmaxf(p.Y, yl(i).x);
#pragma unroll UNROLL
  for (int i = 0; i < n; ++i) {
    const float2 a = yl(i);
    const float4 x = v(i);
    const float f = ex2(a.x - p.Y);
    p.l = fmaf(a.y, f, p.l);
    p.v.x = fmaf(x.x, f, p.v.x), p.v.y = fmaf(x.y, f, p.v.y), p.v.z = fmaf(x.z, f, p.v.z), p.v.w = fmaf(x.w, f, p.v.w);
  }
  return p;
}

// 4 elements of a finished row, and (d0 == 0) its lse.
__device__ __forceinline__ void store_row(const AttendView &a, const Part &p, int64_t row, int DH, int d0) {
  const bool none = p.l == 0.f;  // (a NaN is not)
  const float inv = none ? 0.f : 1.f / p.l;
  *reinterpret_cast<uint2 *>(a.out + row * DH + d0) =
      make_uint2(bf16x2(p.v.x * inv, p.v.y * inv), bf16x2(p.v.z * inv, p.v.w * inv));
  if (a.lse && d0 == 0) a.lse[row] = none ? NEG_INF : (p.Y + log2f(p.l)) * LN2;
}

// every thread of every CTA of the cluster; shared-memory writes before it are
// seen by the reads after it
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// the shared memory of CTA `rank` of the cluster, at this CTA's p
__device__ __forceinline__ uint32_t cluster_at(const void *p, uint32_t rank) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  return at;
}
__device__ __forceinline__ float4 ld_cluster4(const void *p, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_at(p, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(const void *p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_at(p, rank)) : "memory");
  return v;
}

// attend_umma.cu: the same attention for tiles of many rows (heads of a query,
// or of neighbouring queries of one sequence) on tcgen05 tensor cores.  per: queries per tile; tiles: CTAs in x (each goes on by that many).
cudaError_t launch_attend_umma(const KvView &c, const AttendView &a, const Split &sp, int per, int tiles,
                               cudaStream_t s);

}  // namespace misa
