// Rotary positions of up to four tensors of rows in one launch
// (misa_apply_rope).
//
//   (a, b) -> (m (a cos t - b sin t), m (b cos t + a sin t)),  t = p f_i
//
// Bound by the row traffic: every element is read and written once.  A thread
// owns 8 pairs of a row's position (two 16-byte chunks in either layout),
// computes their cos and sin once and applies them to several heads, so the
// arithmetic of the angles (8 sincospif) is spread over 32 bytes x heads.
//
// Measured: 2048 rows of 64 heads of 128 and 2048 single rows, all rotated
// (68 MB): 13.9 us a call in a row of them, 4.9 TB/s, and 16.4 alone in a graph (a
// head at a time, its loads behind the angles: 26.7); issue slots 56 % busy, the
// rest waits for loads.  8 rows: 2.4 us in a row, 4.1 alone, a launch and three
// dependent loads.
#include "attention.h"
#include "rope.cuh"

namespace misa {
namespace {

constexpr int THREADS = 128;

struct Group {
  const uint16_t *x;
  uint16_t *y;
  const int32_t *pos;
  int64_t x_row, x_head, y_row, y_head;
  int n, H, d;
  int units;        // threads per (row, head group)
  int head_groups;  // a row's heads are dealt to this many threads per unit
  int vec;          // 16-byte chunks; else one pair or kept element per unit
  int block0;       // first block of the group
};

struct Groups {
  Group g[MISA_MAX_ROPE_GROUPS];
  int n;
};

__global__ void __launch_bounds__(THREADS, 5) rope_kernel(RopeView r, Groups gs) {
  grid_dep_sync();
  int w = 0;
  while (w + 1 < gs.n && (int)blockIdx.x >= gs.g[w + 1].block0) ++w;
  const Group &g = gs.g[w];
  const int64_t t = (int64_t)((int)blockIdx.x - g.block0) * THREADS + threadIdx.x;
  int u, hg;
  int64_t row;
  if (t >> 31) {
    u = (int)(t % g.units);
    hg = (int)(t / g.units % g.head_groups);
    row = t / g.units / g.head_groups;
  } else {  // (64-bit divisions cost more than the rest of a small row)
    const uint32_t rest = (uint32_t)t / (uint32_t)g.units;
    u = (int)((uint32_t)t - rest * g.units);
    const uint32_t r = rest / (uint32_t)g.head_groups;
    hg = (int)(rest - r * g.head_groups);
    row = r;
  }
  if (row >= g.n) return;
  const int p = g.pos[row];
  const bool in_place = g.x == g.y;
  const uint16_t *x = g.x + row * g.x_row;
  uint16_t *y = g.y + row * g.y_row;
  if (g.vec) {
    int o1, o2;
    const bool rotated = rope_unit(u, g.d, r.rot, r.first, r.interleaved, o1, o2);
    if (!rotated && in_place) return;
    if (!rotated) {
      for (int h = hg; h < g.H; h += g.head_groups) {
        const uint4 a = *reinterpret_cast<const uint4 *>(x + h * g.x_head + o1);
        *reinterpret_cast<uint4 *>(y + h * g.y_head + o1) = a;
        if (o2 >= 0)
          *reinterpret_cast<uint4 *>(y + h * g.y_head + o2) = *reinterpret_cast<const uint4 *>(x + h * g.x_head + o2);
      }
      return;
    }
    // four heads' chunks are on their way while the angles are worked out
    constexpr int AHEAD = 4;
    float2 cs[8];
    bool first = true;
    for (int h = hg; h < g.H; h += AHEAD * g.head_groups) {
      uint4 in[AHEAD][2];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int hh = h + i * g.head_groups;
        if (hh >= g.H) break;
        in[i][0] = *reinterpret_cast<const uint4 *>(x + hh * g.x_head + o1);
        in[i][1] = *reinterpret_cast<const uint4 *>(x + hh * g.x_head + o2);
      }
      if (first) rope_unit_cs(r.phase, u, p, r.amplitude, cs);
      first = false;
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int hh = h + i * g.head_groups;
        if (hh >= g.H) break;
        float a[8], b[8];
        unpack8(in[i][0], a);
        unpack8(in[i][1], b);
        rope_unit_rotate(a, b, cs, r.interleaved);
        *reinterpret_cast<uint4 *>(y + hh * g.y_head + o1) = pack8(a);
        *reinterpret_cast<uint4 *>(y + hh * g.y_head + o2) = pack8(b);
      }
    }
    return;
  }
  if (u < r.rot / 2) {
    const int ea = r.first + (r.interleaved ? 2 * u : u), eb = r.interleaved ? ea + 1 : ea + r.rot / 2;
    const float2 cs = rope_cos_sin(__ldg(r.phase + u), p, r.amplitude);
    for (int h = hg; h < g.H; h += g.head_groups) {
      const uint16_t *xh = x + h * g.x_head;
      uint16_t *yh = y + h * g.y_head;
      const float2 z = rope_pair(bf16_bits_to_float(xh[ea]), bf16_bits_to_float(xh[eb]), cs);
      const uint32_t v = pack_bf16(z.x, z.y);
      yh[ea] = (uint16_t)v;
      yh[eb] = (uint16_t)(v >> 16);
    }
  } else if (!in_place) {
    const int c = u - r.rot / 2, e = c < r.first ? c : c + r.rot;
    for (int h = hg; h < g.H; h += g.head_groups) y[h * g.y_head + e] = x[h * g.x_head + e];
  }
}

bool on16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

cudaError_t launch_rope(const RopeView &r, const misa_rope_rows *groups, int n_groups, cudaStream_t s) {
  Groups gs = {};
  int64_t blocks = 0;
  for (int i = 0; i < n_groups; ++i) {
    const misa_rope_rows &q = groups[i];
    if (q.n == 0 || q.H == 0) continue;
    Group &g = gs.g[gs.n++];
    g.x = q.x, g.y = q.y, g.pos = q.pos;
    g.x_row = q.x_row, g.x_head = q.x_head, g.y_row = q.y_row, g.y_head = q.y_head;
    g.n = q.n, g.H = q.H, g.d = q.d;
    g.vec = r.rot % 16 == 0 && r.first % 8 == 0 && q.d % 8 == 0 && on16(q.x) && on16(q.y) && q.x_row % 8 == 0 &&
            q.x_head % 8 == 0 && q.y_row % 8 == 0 && q.y_head % 8 == 0;
    g.units = g.vec ? r.rot / 16 + cdiv(q.d - r.rot, 16) : r.rot / 2 + (q.d - r.rot);
    const int per = heads_per_thread((int64_t)q.n * g.units * q.H, q.H);
    g.head_groups = cdiv(q.H, per);
    g.block0 = (int)blocks;
    blocks += ((int64_t)q.n * g.head_groups * g.units + THREADS - 1) / THREADS;
  }
  if (blocks == 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  return launch_kernel(rope_kernel, dim3((unsigned)blocks), dim3(THREADS), 0, s, r, gs);
}

}  // namespace misa
