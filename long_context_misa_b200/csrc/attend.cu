// Attention over each query's selected tokens, or its whole prefix, with a
// tree of drafted tokens behind it (misa_attend).
//
//   s_t = scale q.k_t,  out = sum_t e^(s_t) v_t / sum_t e^(s_t),
//   lse = ln sum_t e^(s_t)    over the tokens t that the query sees
//
// One pass over the tokens with a running maximum and sum per row (a row is a
// head of a query).  The G = H / H_kv heads that read one key/value head are
// the rows of a matrix tile, so a token's key and value are fetched once for
// all of them: bound by the rows' bytes (e4m3, d = 128: 264 bytes per token
// and key/value head against 4 G d flops) for the few rows of decode.
//
// attend_kernel: a CTA of 8 warps holds 16 MT rows of one key/value head and
// a share of the tokens (blockIdx.z of Z shares).  Each warp runs alone
// through every 8th chunk of CH tokens: it gathers the rows with 16-byte
// cp.async into its own ring of STAGES chunks, so no barrier sits in the loop
// and about 128 KB of rows are in flight per SM.  S = Q K^T and O += P V are
// mma.sync m16n8k16 with fp32 sums.  The 8 warps' (max, sum, O) meet in shared
// memory at the end; with Z > 1 the CTAs' meet in the workspace, where
// attend_combine_kernel joins them in a fixed order.
//
// Numbers.  bf16 caches: bf16 products; the weights e^(s - max) are rounded to
// bf16 before they meet the values.  e4m3 caches: codes are exact in f16; a
// query row is scaled by a power of two into f16's range (bf16 has 8
// significant bits, so elements down to 2^-24 of the row's largest stay
// exact); the weights of the sum are e^(s_t - max s) in fp32, and what meets
// the value codes is e^(s_t - max s) v_scale_t 2^-c <= 1 in f16, with c the
// running maximum of log2 of the contributions (relative to max s): so the
// largest contribution of a row sets f16's range, not the largest scale.
#include <algorithm>

#include "attention.h"

namespace misa {
namespace {

constexpr int NW = 8;  // warps per CTA
constexpr int THREADS = NW * 32;
constexpr int STAGES = 3;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float NEG_INF = -__builtin_huge_valf();

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// 2^(7 - E) for amax = m 2^E, m in [0.5, 1): the row's largest element lands
// in [64, 128).  1 for rows of zeros or with a NaN or infinity.
__device__ __forceinline__ float row_scale(float amax) {
  if (!(amax > 0.f) || !isfinite(amax)) return 1.f;
  const int e = 7 - ((int)(__float_as_uint(amax) >> 23) - 126);
  return ldexpf(1.f, min(max(e, -126), 126));
}

template <int DH, bool FP8>
struct Cfg {
  static constexpr int CH = FP8 ? 32 : 16;          // tokens per chunk
  static constexpr int RB = DH * (FP8 ? 1 : 2);     // bytes per row
  static constexpr int CPR = RB / 16;               // 16-byte pieces per row
  static constexpr int KT = DH / 16;                // k-tiles of S
  static constexpr int NT = CH / 8;                 // token n-tiles of S
  static constexpr int VT = DH / 8;                 // value n-tiles of O
  static constexpr int STAGE = 2 * CH * RB + (FP8 ? 2 * CH * 4 : 0) + 16;  // keys, values, scales, mask word
};

// Piece `c` of row `r`: keys are read as 16-byte pieces of two neighbouring
// rows per quarter warp, values by ldmatrix over 8 rows; both without bank
// conflicts under these permutations.
template <int RB>
__device__ __forceinline__ int k_piece(int r, int c) {
  return RB >= 128 ? c ^ ((r & 1) << 2) : c;
}
template <int RB>
__device__ __forceinline__ int v_piece(int r, int c) {
  return RB >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
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

// The queries of a CTA's rows that share a sequence, and the chunks of its
// prefix and drafted tokens.
struct Run {
  int seq, len;      // longest prefix of its rows
  int row0, row1;    // rows of the CTA
  int c0, c1, c2;    // chunks [c0, c1): prefix, [c1, c2): drafted
  int draft0;        // position of drafted slot 0
};

template <int MT>
struct RowInfo {
  int len[16 * MT];    // prefix length (0 for rows that hold nothing)
  int query[16 * MT];  // -1: no such row
};

struct Split {
  float *o;      // [Z][n_q * H][DH]
  float4 *ml;    // [Z][n_q * H] (max, sum, reference of O)
  int Z;
};

template <int DH, bool FP8, int MT, bool LIST>
__global__ void __launch_bounds__(THREADS, 1)
    attend_kernel(KvView c, AttendView a, Split split, int tiles_per_query) {
  grid_dep_sync();
  using F = Cfg<DH, FP8>;
  constexpr int R = 16 * MT, CH = F::CH, RB = F::RB;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ RowInfo<MT> rows;
  __shared__ Run runs[R];
  __shared__ int n_runs_s;
  __shared__ __align__(16) uint4 qfrag[MT * F::KT * 32];
  __shared__ float row_mul[R];  // scale log2(e) over the row's power of two

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c4 = lane & 3;
  const int G = a.H / c.H_kv, hk = blockIdx.y, Z = split.Z;
  const int tile = blockIdx.x;
  // row r of the CTA -> query and head
  const int q0 = LIST ? tile / tiles_per_query : 0;
  const int g0 = LIST ? (tile % tiles_per_query) * R : 0;
  auto row_query = [&](int r) -> int {
    if (LIST) return g0 + r < G ? q0 : -1;
    const int64_t x = (int64_t)tile * R + r;
    return x < (int64_t)a.n_q * G ? (int)(x / G) : -1;
  };
  auto row_head = [&](int r) -> int {
    return hk * G + (LIST ? g0 + r : (int)(((int64_t)tile * R + r) % G));
  };

  // ---- rows, runs ----
  __shared__ int row_seq[R];
  if (tid < R) {
    const int q = row_query(tid);
    int s = -1, len = 0;
    if (q >= 0) len = attend_prefix(c, a, q, &s);
    rows.query[tid] = q;
    rows.len[tid] = len;
    row_seq[tid] = s;
  }
  __syncthreads();
  if (tid == 0) {
    int n = 0, chunks = 0;
    for (int r = 0; r < R;) {
      if (row_seq[r] < 0) {
        ++r;
        continue;
      }
      Run u;
      u.seq = row_seq[r];
      u.row0 = r;
      u.len = 0;
      while (r < R && row_seq[r] == u.seq) u.len = max(u.len, rows.len[r++]);
      u.row1 = r;
      u.c0 = chunks;
      chunks += LIST ? cdiv(a.k, CH) : cdiv(u.len, CH);
      u.c1 = chunks;
      u.draft0 = 0;
      if (a.draft_start) {
        chunks += cdiv(a.n_draft, CH);
        u.draft0 = a.draft_start[u.seq];
      }
      u.c2 = chunks;
      runs[n++] = u;
    }
    n_runs_s = n;
  }
  // ---- query fragments: the k dimension permuted so that a 16-byte piece of
  // a key row feeds whole B fragments (see tile loop) ----
  for (int r = warp; r < R; r += NW) {
    const int q = row_query(r);
    float sc = 1.f;
    if (FP8) {
      float m = 0.f;
      if (q >= 0) {
        const uint16_t *src = a.q + ((int64_t)q * a.H + row_head(r)) * DH;
        for (int e = lane; e < DH; e += 32) {
          const float x = fabsf(bf16_bits_to_float(src[e]));
          m = (x > m || x != x) ? x : m;  // a NaN stays
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const float x = __shfl_xor_sync(0xffffffffu, m, o);
        m = (x > m || x != x) ? x : m;
      }
      sc = row_scale(m);
    }
    if (lane == 0) row_mul[r] = sc;
  }
  __syncthreads();
  for (int e = tid; e < MT * F::KT * 32; e += THREADS) {
    const int l = e & 31, kt = (e >> 5) % F::KT, mt = (e >> 5) / F::KT;
    // FP8: piece of 16 elements feeds 4 k-tiles; bf16: of 8 elements, 2
    const int ch = FP8 ? kt >> 2 : kt >> 1, u = FP8 ? kt & 3 : kt & 1;
    const int d0 = FP8 ? 64 * ch + 16 * (l & 3) + 4 * u : 32 * ch + 8 * (l & 3) + 4 * u;
    uint32_t w[4];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = mt * 16 + (l >> 2) + 8 * half;
      const int q = row_query(r);
      uint2 v = make_uint2(0u, 0u);
      if (q >= 0) v = *reinterpret_cast<const uint2 *>(a.q + ((int64_t)q * a.H + row_head(r)) * DH + d0);
      if (FP8) {
        const float sc = row_mul[r];
        const float2 x = bf16x2_to_float2(v.x), y = bf16x2_to_float2(v.y);
        v.x = f16x2(x.x * sc, x.y * sc);
        v.y = f16x2(y.x * sc, y.y * sc);
      }
      w[half] = v.x;
      w[2 + half] = v.y;
    }
    qfrag[e] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncthreads();
  if (tid < R) row_mul[tid] = a.scale * LOG2E / row_mul[tid];
  __syncthreads();

  // ---- this CTA's chunks, every NW-th to a warp ----
  const int n_runs = n_runs_s;
  const int chunks = n_runs ? runs[n_runs - 1].c2 : 0;
  const int share = cdiv(chunks, Z);
  const int cb = min((int)blockIdx.z * share, chunks), ce = min(cb + share, chunks);

  float o[MT][F::VT][4];
  // base 2: running maximum of the logits, sum of the weights relative to it,
  // and the exponent that O is relative to (bf16 caches: the maximum itself)
  float m_run[MT][2], l_run[MT][2], y_run[MT][2];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int n = 0; n < F::VT; ++n) o[mt][n][0] = o[mt][n][1] = o[mt][n][2] = o[mt][n][3] = 0.f;
    m_run[mt][0] = m_run[mt][1] = y_run[mt][0] = y_run[mt][1] = NEG_INF;
    l_run[mt][0] = l_run[mt][1] = 0.f;
  }

  uint8_t *ring = smem + warp * (STAGES * F::STAGE);
  auto stage_k = [&](int st) { return ring + st * F::STAGE; };
  auto stage_v = [&](int st) { return ring + st * F::STAGE + CH * RB; };
  auto stage_s = [&](int st) { return reinterpret_cast<float *>(ring + st * F::STAGE + 2 * CH * RB); };
  auto stage_m = [&](int st) {
    return reinterpret_cast<uint32_t *>(ring + st * F::STAGE + F::STAGE - 16);
  };

  // Position of this lane's token of a chunk (lane < CH), -1 for none.
  int run_i = 0;  // run of the chunk last asked for (chunks ascend)
  auto token_of = [&](int ck) -> int {
    if (ck >= ce) return -1;
    while (ck >= runs[run_i].c2) ++run_i;
    const Run &u = runs[run_i];
    const int l = lane & (CH - 1);
    if (ck >= u.c1) {
      const int j = (ck - u.c1) * CH + l;
      if (j >= a.n_draft) return -1;
      bool want = true;
      if (LIST) want = (a.draft_mask[(int64_t)q0 * cdiv(a.n_draft, 32) + (j >> 5)] >> (j & 31)) & 1u;
      if (!want) return -1;
      const int64_t p = (int64_t)u.draft0 + j;
      if (p >= 0 && p < c.L_cap) return (int)p;
      if (LIST) flag(c, MISA_DEV_BAD_POSITION);
      return -1;
    }
    const int t = (ck - u.c0) * CH + l;
    if (!LIST) return t < u.len ? t : -1;
    if (t >= a.k) return -1;
    const int tok = __ldg(a.topk + (int64_t)q0 * a.k + t);
    return tok >= 0 && tok < u.len ? tok : -1;
  };
  // Gather chunk rows into stage st.
  auto issue = [&](int st, int ck, int tok) {
    if (ck < ce) {
      const uint32_t have = __ballot_sync(0xffffffffu, tok >= 0);
      const int64_t base = (int64_t)runs[run_i].seq * c.L_cap;
      if (have) {
        const uint32_t sk = smem_addr(stage_k(st)), sv = smem_addr(stage_v(st));
#pragma unroll
        for (int it = 0; it < CH * F::CPR / 32; ++it) {
          const int r = it * (32 / F::CPR) + lane / F::CPR, pc = lane % F::CPR;
          const int t = __shfl_sync(0xffffffffu, tok, r);
          const int64_t off = ((base + max(t, 0)) * c.H_kv + hk) * RB + pc * 16;
          cp_async16(sk + r * RB + k_piece<RB>(r, pc) * 16, c.k + off, t >= 0);
          cp_async16(sv + r * RB + v_piece<RB>(r, pc) * 16, c.v + off, t >= 0);
        }
        if (FP8 && lane < CH) {
          const int64_t row = (base + max(tok, 0)) * c.H_kv + hk;
          const uint32_t ss = smem_addr(stage_s(st));
          cp_async4(ss + lane * 4, c.k_scale + row, tok >= 0);
          cp_async4(ss + (CH + lane) * 4, c.v_scale + row, tok >= 0);
        }
      }
      if (lane == 0) *stage_m(st) = CH == 32 ? have : have & 0xFFFFu;
    }
    cp_async_commit();
  };

  int nxt = cb + warp;  // next chunk to issue
  int tok_n = token_of(nxt);
#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st) {
    issue(st, nxt, tok_n);
    nxt += NW;
    tok_n = token_of(nxt);
  }
  int st = 0, run_c = 0;
  for (int ck = cb + warp; ck < ce; ck += NW) {
    cp_async_wait<STAGES - 2>();
    __syncwarp();
    const int wr = st == 0 ? STAGES - 1 : st - 1;
    const uint32_t have = *stage_m(st);
    // (the stage written now was last read in the iteration before; the
    // __syncwarp above orders those reads)
    issue(wr, nxt, tok_n);
    nxt += NW;
    tok_n = token_of(nxt);
    const uint8_t *sk = stage_k(st), *sv = stage_v(st);
    const float *ss = stage_s(st);
    st = st == STAGES - 1 ? 0 : st + 1;
    if (!have) continue;
    while (ck >= runs[run_c].c2) ++run_c;
    const Run &u = runs[run_c];

    // ---- S = Q K^T ----
    float s[MT][F::NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int n = 0; n < F::NT; ++n) s[mt][n][0] = s[mt][n][1] = s[mt][n][2] = s[mt][n][3] = 0.f;
#pragma unroll
    for (int ch = 0; ch < RB / 64; ++ch) {
      uint4 kv[F::NT];
#pragma unroll
      for (int n = 0; n < F::NT; ++n) {
        const int r = n * 8 + g;
        kv[n] = *reinterpret_cast<const uint4 *>(sk + r * RB + k_piece<RB>(r, 4 * ch + c4) * 16);
      }
#pragma unroll
      for (int uu = 0; uu < (FP8 ? 4 : 2); ++uu) {
        const int kt = ch * (FP8 ? 4 : 2) + uu;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint4 qf = qfrag[(mt * F::KT + kt) * 32 + lane];
          const uint32_t af[4] = {qf.x, qf.y, qf.z, qf.w};
#pragma unroll
          for (int n = 0; n < F::NT; ++n) {
            if (FP8) {
              const uint32_t w = uu == 0 ? kv[n].x : uu == 1 ? kv[n].y : uu == 2 ? kv[n].z : kv[n].w;
              mma_f16_16816(s[mt][n], af, e4m3x2_to_f16x2((uint16_t)w), e4m3x2_to_f16x2((uint16_t)(w >> 16)));
            } else {
              mma_bf16_16816(s[mt][n], af, uu ? kv[n].z : kv[n].x, uu ? kv[n].w : kv[n].y);
            }
          }
        }
      }
    }

    // ---- visible tokens, scales, running maximum ----
    float lv[F::NT][2], vs[F::NT][2], ks[F::NT][2];
    if (FP8) {
#pragma unroll
      for (int n = 0; n < F::NT; ++n) {
        const float2 kk = *reinterpret_cast<const float2 *>(ss + n * 8 + 2 * c4);
        const float2 vv = *reinterpret_cast<const float2 *>(ss + CH + n * 8 + 2 * c4);
        ks[n][0] = kk.x, ks[n][1] = kk.y;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          vs[n][x] = x ? vv.y : vv.x;
          lv[n][x] = __log2f(vs[n][x] < 0x1p-100f ? 0x1p-100f : vs[n][x]);  // a NaN stays
        }
      }
    }
    uint32_t vis[MT][2];
    bool mixed = false;  // some row does not see a gathered token
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int r = mt * 16 + g + 8 * hf;
        if (LIST) {
          vis[mt][hf] = rows.query[r] >= 0 ? have : 0u;
        } else {
          uint32_t v = 0u;
          if (r >= u.row0 && r < u.row1) {
            if (ck < u.c1) {
              const int nn = rows.len[r] - (ck - u.c0) * CH;
              v = nn >= 32 ? 0xffffffffu : nn > 0 ? (1u << nn) - 1u : 0u;
            } else {
              const int j0 = (ck - u.c1) * CH;
              v = a.draft_mask[(int64_t)rows.query[r] * cdiv(a.n_draft, 32) + (j0 >> 5)] >> (j0 & 31);
              if (CH < 32) v &= (1u << CH) - 1u;
              if ((a.n_draft - j0) < CH) v &= (1u << (a.n_draft - j0)) - 1u;
              if ((v & ~have) && c4 == 0) flag(c, MISA_DEV_BAD_POSITION);
            }
          }
          vis[mt][hf] = v & have;
          mixed |= vis[mt][hf] != have;
        }
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const float mul = row_mul[mt * 16 + g + 8 * hf];
        float mx = NEG_INF, my = NEG_INF;
#pragma unroll
        for (int n = 0; n < F::NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float &v = s[mt][n][2 * hf + x];
            v = FP8 ? v * ks[n][x] * mul : v * mul;
            if (!((vis[mt][hf] >> (n * 8 + 2 * c4 + x)) & 1u)) v = NEG_INF;
            mx = fmaxf(mx, v);
            if (FP8) my = fmaxf(my, v + lv[n][x]);
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        if (FP8) {
          my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 1));
          my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, 2));
        } else {
          my = mx;
        }
        const float m_new = fmaxf(m_run[mt][hf], mx), y_new = fmaxf(y_run[mt][hf], my);
        const float ref = m_new == NEG_INF ? 0.f : m_new, yref = y_new == NEG_INF ? 0.f : y_new;
        if (m_new != m_run[mt][hf]) {
          l_run[mt][hf] *= ex2(m_run[mt][hf] - ref);
          m_run[mt][hf] = m_new;
        }
        if (y_new != y_run[mt][hf]) {
          const float al = ex2(y_run[mt][hf] - yref);
#pragma unroll
          for (int n = 0; n < F::VT; ++n) {
            o[mt][n][2 * hf] *= al;
            o[mt][n][2 * hf + 1] *= al;
          }
          y_run[mt][hf] = y_new;
        }
        const float f = FP8 ? ex2(ref - yref) : 1.f;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < F::NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float &v = s[mt][n][2 * hf + x];
            const bool seen = LIST || v != NEG_INF;
            v = ex2(v - ref);
            sum += v;
            // (gathered rows that this one does not see may hold any scale)
            if (FP8) v = seen ? v * (vs[n][x] * f) : 0.f;
          }
        l_run[mt][hf] += sum;
      }

    // ---- values that some rows must not see: a NaN or infinity there would
    // reach them as 0 * NaN.  Such values are taken out of the tile and added
    // to the rows that do see them ----
    if (!LIST && __any_sync(0xffffffffu, mixed)) {
      for (int e = lane; e < CH * RB / 4; e += 32) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(sv)[e];
        bool bad;
        if (FP8)
          bad = (__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu)) != 0u;
        else
          bad = (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
        uint32_t who = __ballot_sync(0xffffffffu, bad);
        while (who) {
          const int src = __ffs(who) - 1;
          who &= who - 1;
          const int be = e - lane + src;  // word of the tile
          const uint32_t bw = __shfl_sync(0xffffffffu, w, src);
          const int r = be / (RB / 4), off = (be % (RB / 4)) * 4;
          const int pc = v_piece<RB>(r, off >> 4);  // the permutation is its own inverse
          for (int b = 0; b < (FP8 ? 4 : 2); ++b) {
            const uint32_t el = FP8 ? (bw >> (8 * b)) & 0xffu : (bw >> (16 * b)) & 0xffffu;
            if (FP8 ? (el & 0x7fu) != 0x7fu : (el & 0x7f80u) != 0x7f80u) continue;
            const float val = FP8 ? __int_as_float(0x7fffffff) : bf16_bits_to_float(el);
            const int dd = FP8 ? pc * 16 + (off & 15) + b : (pc * 16 + (off & 15)) / 2 + b;
            // accumulator of element dd: n-tile and register of its lane
            const int n_of = FP8 ? 2 * (dd >> 4) + (dd & 1) : dd >> 3;
            const int col = FP8 ? (dd & 15) >> 1 : dd & 7;  // column of the n-tile
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                float wt = 0.f;
#pragma unroll
                for (int n = 0; n < F::NT; ++n)
#pragma unroll
                  for (int x = 0; x < 2; ++x)
                    if (n == (r >> 3) && x == (r & 1)) wt = s[mt][n][2 * hf + x];
                wt = __shfl_sync(0xffffffffu, wt, (lane & ~3) | ((r & 7) >> 1));
                if (c4 == col >> 1 && ((vis[mt][hf] >> r) & 1u)) {
#pragma unroll
                  for (int n = 0; n < F::VT; ++n)
                    if (n == n_of) o[mt][n][2 * hf + (col & 1)] += wt * val;
                }
              }
          }
          if (lane == src) {
            uint32_t z = bw;
            if (FP8) {
              for (int b = 0; b < 4; ++b)
                if (((bw >> (8 * b)) & 0x7fu) == 0x7fu) z &= ~(0xffu << (8 * b));
            } else {
              if ((bw & 0x7f80u) == 0x7f80u) z &= 0xffff0000u;
              if ((bw & 0x7f800000u) == 0x7f800000u) z &= 0xffffu;
            }
            reinterpret_cast<uint32_t *>(const_cast<uint8_t *>(sv))[be] = z;
          }
        }
      }
      __syncwarp();
    }

    // ---- O += P V ----
#pragma unroll
    for (int tk = 0; tk < CH / 16; ++tk) {
      uint32_t pf[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const float(&x)[4] = s[mt][2 * tk];
        const float(&y)[4] = s[mt][2 * tk + 1];
        pf[mt][0] = FP8 ? f16x2(x[0], x[1]) : bf16x2(x[0], x[1]);
        pf[mt][1] = FP8 ? f16x2(x[2], x[3]) : bf16x2(x[2], x[3]);
        pf[mt][2] = FP8 ? f16x2(y[0], y[1]) : bf16x2(y[0], y[1]);
        pf[mt][3] = FP8 ? f16x2(y[2], y[3]) : bf16x2(y[2], y[3]);
      }
      const int mtx = lane >> 3, vr = tk * 16 + (mtx & 1) * 8 + (lane & 7);
#pragma unroll
      for (int j = 0; j < F::CPR / 2; ++j) {
        uint32_t r[4];
        ldmatrix_x4_trans(r, smem_addr(sv + vr * RB + v_piece<RB>(vr, 2 * j + (mtx >> 1)) * 16));
        if (FP8) {
          // a register holds elements (2n, 2n+1) of tokens 2c and 2c+1: the
          // even ones form one n-tile, the odd ones the next
#pragma unroll
          for (int dg = 0; dg < 2; ++dg) {
            const uint32_t b0 = __byte_perm(r[2 * dg], 0, 0x3120), b1 = __byte_perm(r[2 * dg + 1], 0, 0x3120);
            const uint32_t e0 = e4m3x2_to_f16x2((uint16_t)b0), e1 = e4m3x2_to_f16x2((uint16_t)b1);
            const uint32_t o0 = e4m3x2_to_f16x2((uint16_t)(b0 >> 16)), o1 = e4m3x2_to_f16x2((uint16_t)(b1 >> 16));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              mma_f16_16816(o[mt][4 * j + 2 * dg], pf[mt], e0, e1);
              mma_f16_16816(o[mt][4 * j + 2 * dg + 1], pf[mt], o0, o1);
            }
          }
        } else {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma_bf16_16816(o[mt][2 * j], pf[mt], r[0], r[1]);
            mma_bf16_16816(o[mt][2 * j + 1], pf[mt], r[2], r[3]);
          }
        }
      }
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // every ring is free: its memory takes the warps' results

  // ---- join the warps ----
  float *so = reinterpret_cast<float *>(smem);                              // [NW][R][DH]
  float4 *sml = reinterpret_cast<float4 *>(smem + (size_t)NW * R * DH * 4);  // [NW][R]
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float l = l_run[mt][hf];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int r = mt * 16 + g + 8 * hf;
      if (c4 == 0) sml[warp * R + r] = make_float4(m_run[mt][hf], l, y_run[mt][hf], 0.f);
      float *row = so + ((size_t)warp * R + r) * DH;
#pragma unroll
      for (int n = 0; n < F::VT; ++n) {
        if (FP8) {
          // n-tiles 2j and 2j+1: elements 16j + 4c4 + {0, 2} and {1, 3}
          if ((n & 1) == 0)
            *reinterpret_cast<float4 *>(row + 8 * n + 4 * c4) =
                make_float4(o[mt][n][2 * hf], o[mt][n | 1][2 * hf], o[mt][n][2 * hf + 1], o[mt][n | 1][2 * hf + 1]);
        } else {
          *reinterpret_cast<float2 *>(row + 8 * n + 2 * c4) = make_float2(o[mt][n][2 * hf], o[mt][n][2 * hf + 1]);
        }
      }
    }
  __syncthreads();
  for (int e = tid; e < R * (DH / 4); e += THREADS) {
    const int r = e / (DH / 4), d0 = (e % (DH / 4)) * 4;
    const int q = rows.query[r];
    if (q < 0) continue;
    float M = NEG_INF, Y = NEG_INF;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      M = fmaxf(M, sml[w * R + r].x);
      Y = fmaxf(Y, sml[w * R + r].z);
    }
    const float ref = M == NEG_INF ? 0.f : M, yref = Y == NEG_INF ? 0.f : Y;
    float l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float4 ml = sml[w * R + r];
      const float f = ex2(ml.z - yref);
      const float4 x = *reinterpret_cast<const float4 *>(so + ((size_t)w * R + r) * DH + d0);
      l = fmaf(ml.y, ex2(ml.x - ref), l);
      v.x = fmaf(x.x, f, v.x), v.y = fmaf(x.y, f, v.y), v.z = fmaf(x.z, f, v.z), v.w = fmaf(x.w, f, v.w);
    }
    const int64_t orow = (int64_t)q * a.H + row_head(r);
    if (Z > 1) {
      const int64_t prow = (int64_t)blockIdx.z * a.n_q * a.H + orow;
      *reinterpret_cast<float4 *>(split.o + prow * DH + d0) = v;
      if (d0 == 0) split.ml[prow] = make_float4(M, l, Y, 0.f);
    } else {
      const bool none = M == NEG_INF && l == 0.f;
      const float inv = none ? 0.f : ex2(yref - ref) / l;
      *reinterpret_cast<uint2 *>(a.out + orow * DH + d0) =
          make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
      if (a.lse && d0 == 0) a.lse[orow] = none ? NEG_INF : M * LN2 + logf(l);
    }
  }
}

// One warp per row: the Z shares' (max, sum, O), joined in order.
template <int DH>
__global__ void __launch_bounds__(128) attend_combine_kernel(AttendView a, Split split) {
  grid_dep_sync();
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), n = (int64_t)a.n_q * a.H;
  const int lane = threadIdx.x & 31;
  if (row >= n) return;
  float M = NEG_INF, Y = NEG_INF;
  for (int z = lane; z < split.Z; z += 32) {
    const float4 ml = split.ml[z * n + row];
    M = fmaxf(M, ml.x);
    Y = fmaxf(Y, ml.z);
  }
#pragma unroll
  for (int x = 16; x; x >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    Y = fmaxf(Y, __shfl_xor_sync(0xffffffffu, Y, x));
  }
  const float ref = M == NEG_INF ? 0.f : M, yref = Y == NEG_INF ? 0.f : Y;
  constexpr int E = DH / 32;
  float v[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = 0.f;
  for (int z = 0; z < split.Z; ++z) {
    const float4 ml = split.ml[z * n + row];
    const float f = ex2(ml.z - yref);
    l = fmaf(ml.y, ex2(ml.x - ref), l);
    const float *p = split.o + (z * n + row) * DH + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = fmaf(p[e], f, v[e]);
  }
  const bool none = M == NEG_INF && l == 0.f;
  const float inv = none ? 0.f : ex2(yref - ref) / l;
  uint32_t *out = reinterpret_cast<uint32_t *>(a.out + row * DH + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = bf16x2(v[e] * inv, v[e + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = none ? NEG_INF : M * LN2 + logf(l);
}

struct Plan {
  int mt, tiles, tiles_per_query, Z;
};

// The most chunks a CTA row tile can have (lengths are on the device: whole
// prefixes count as full caches).
Plan make_plan(int n_q, int H, int H_kv, int L_cap, bool fp8, int k, int n_draft) {
  Plan p;
  const int G = H / H_kv;
  const bool list = k > 0;
  const int64_t rows = list ? G : (int64_t)n_q * G;
  p.mt = rows > 16 ? 2 : 1;
  const int R = 16 * p.mt, CH = fp8 ? 32 : 16;
  p.tiles_per_query = list ? cdiv(G, R) : 0;
  p.tiles = list ? n_q * p.tiles_per_query : (int)((rows + R - 1) / R);
  const int chunks = cdiv(list ? k : L_cap, CH) + cdiv(n_draft, CH);
  const int64_t ctas = (int64_t)p.tiles * H_kv;
  // shares: fill the SMs once, two chunks per warp at the least
  const int64_t want = ctas > 0 ? device_sms() / ctas : 1;
  p.Z = (int)std::max<int64_t>(1, std::min<int64_t>(want, chunks / (2 * NW)));
  return p;
}

template <int DH, bool FP8, int MT, bool LIST>
cudaError_t run_attend(const KvView &c, const AttendView &a, const Split &sp, const Plan &p, cudaStream_t s) {
  using F = Cfg<DH, FP8>;
  constexpr size_t ring = (size_t)NW * STAGES * F::STAGE, join = (size_t)NW * 16 * MT * (DH * 4 + 16);
  constexpr size_t bytes = ring > join ? ring : join;
  struct Tag {};
  const int have = cached_per_device<Tag>([] { return opt_in_max_dyn_smem(attend_kernel<DH, FP8, MT, LIST>); });
  if (have < (int)bytes) return cudaErrorInvalidConfiguration;
  return launch_kernel(attend_kernel<DH, FP8, MT, LIST>, dim3(p.tiles, c.H_kv, p.Z), dim3(THREADS), bytes, s, c, a, sp,
                       p.tiles_per_query);
}

template <int DH, bool FP8>
cudaError_t pick_attend(const KvView &c, const AttendView &a, const Split &sp, const Plan &p, cudaStream_t s) {
  if (a.topk)
    return p.mt == 2 ? run_attend<DH, FP8, 2, true>(c, a, sp, p, s) : run_attend<DH, FP8, 1, true>(c, a, sp, p, s);
  return p.mt == 2 ? run_attend<DH, FP8, 2, false>(c, a, sp, p, s) : run_attend<DH, FP8, 1, false>(c, a, sp, p, s);
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t attend_ws_bytes(const KvView &c, int n_q, int H, int k, int n_draft) {
  const Plan p = make_plan(n_q, H, c.H_kv, c.L_cap, c.fp8, k, n_draft);
  if (p.Z <= 1) return 0;
  const size_t n = (size_t)p.Z * n_q * H;
  return round256(n * c.d * 4) + round256(n * 16);
}

cudaError_t launch_attend(const KvView &c, const AttendView &a, void *ws, cudaStream_t s) {
  if (a.n_q == 0) return cudaSuccess;
  const Plan p = make_plan(a.n_q, a.H, c.H_kv, c.L_cap, c.fp8, a.topk ? a.k : 0, a.n_draft);
  Split sp = {nullptr, nullptr, p.Z};
  if (p.Z > 1) {
    sp.o = static_cast<float *>(ws);
    sp.ml = reinterpret_cast<float4 *>(static_cast<uint8_t *>(ws) + round256((size_t)p.Z * a.n_q * a.H * c.d * 4));
  }
  cudaError_t e = c.d == 128 ? (c.fp8 ? pick_attend<128, true>(c, a, sp, p, s) : pick_attend<128, false>(c, a, sp, p, s))
                             : (c.fp8 ? pick_attend<64, true>(c, a, sp, p, s) : pick_attend<64, false>(c, a, sp, p, s));
  if (e != cudaSuccess || p.Z == 1) return e;
  const dim3 g((unsigned)(((int64_t)a.n_q * a.H + 3) / 4)), b(128);
  return c.d == 128 ? launch_kernel(attend_combine_kernel<128>, g, b, 0, s, a, sp)
                    : launch_kernel(attend_combine_kernel<64>, g, b, 0, s, a, sp);
}

}  // namespace misa
