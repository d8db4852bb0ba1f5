// Attention over each query's selected tokens, or its whole prefix, with a
// tree of drafted tokens behind it (misa_attend).
//
//   s_t = scale q.k_t,  out = sum_t e^(s_t) v_t / sum_t e^(s_t),
//   lse = ln sum_t e^(s_t)    over the tokens t that the query sees
//
// One pass over the tokens with a running maximum and sum per row (a row is a
// head of a query).  The G = H / H_kv heads that read one key/value head (and,
// without lists, the neighbouring queries of one sequence) are the rows of a
// tile, so a token's key and value are fetched once for all of them.
//
// attend_kernel: a CTA holds up to 8 NR rows of one key/value head and a share
// of the tokens (blockIdx.z of Z shares).  Each warp runs alone through every
// NW-th chunk of 16 or 32 tokens: it gathers the chunk's rows with 16-byte cp.async
// into its own ring of chunks, so no barrier sits in the loop and 100 to
// 130 KB of rows are in flight per SM.  The tokens are the M side of mma.sync
// m16n8k16 (S^T = K Q^T, O^T += V^T P^T), the rows the N side: 8 rows pad
// nothing where M would pad to 16, and a lane keeps two tokens' scales.  P^T
// turns from accumulator to operand by movmatrix.  The maximum is lazy: while
// no weight grows by more than 2^8 nothing is rescaled and no lane exchanges
// anything.
// The warps' (max, sum, O) meet in shared memory at the end.  Up to 8 shares
// are the CTAs of a thread-block cluster and join over its distributed shared
// memory, in a fixed order; more shares meet in the workspace, where
// attend_combine_kernel joins them.
//
// Measured, heads of 128, e4m3, calls one behind the other in a graph.  Lists of
// 2048 tokens, 8 queries x 64 heads on 8 key/value heads: 15.4 us for 35 MB of
// rows (5.3 us of HBM); the lists' look-up and the join of 8 shares come before
// and after them.  512 queries x 64 heads on 4: 183 us for 1.1 GB of gathered
// rows (6.0 TB/s), and 128 x 64 on 8: 80 us for 0.56 GB.  Nothing is saturated
// there (128 queries, captured): L2 21 %, reads over the crossbar 17 %, L1 47 %,
// mma.sync 32 %, issue slots 39 %; a scheduler has 1.8 warps, 0.48 of them
// eligible, and the largest stall is the fixed latency of an instruction.  It is
// the chain of a chunk's steps, with the 8 warps per SM that the registers of O
// leave; forms with more warps, longer chunks and fewer instructions per chunk
// took the same time.  Whole prefixes, 8 x 16K tokens, 4 heads per key/value
// head: 58 us, 4.7 TB/s (bf16: 84 us, 6.4 TB/s).
//
// Numbers.  bf16 caches: bf16 products; the weights e^(s - ref) are rounded to
// bf16 before they meet the values (both sides of a product have one type, and
// a second product for the lower halves would double the products of P V).  e4m3 caches: codes are exact in f16; each
// row of queries is scaled by a power of two of its own into f16's range (bf16
// has 8 significant bits, so elements down to 2^-23 of the row's largest stay
// exact).  With ref 7 binary orders below the running maximum of
// s_t + ln v_scale_t, the sum of the weights e^(s_t - ref) stays in fp32, and
// what meets the value codes is e^(s_t - ref) v_scale_t in f16: a row's largest
// contribution, not its largest scale, sets f16's range, and what it loses is
// 2^-32 of that.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "attend.cuh"

namespace misa {
namespace {

// Tokens per chunk: two m-tiles of e4m3 rows (their widening makes the loop
// bound by instructions, and a longer chunk shares its bookkeeping), one of
// bf16 rows, whose rings take twice the memory, and beside the O of 32 rows.
__host__ __device__ constexpr int chunk_tokens(bool fp8, int nr) { return fp8 && nr == 2 ? 32 : 16; }

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 8 x 8 matrix of 16-bit values across the warp, transposed
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// base + x * BYTES in one instruction
template <int BYTES>
__device__ __forceinline__ const uint8_t *row_at(const uint8_t *base, uint32_t x) {
  uint64_t p;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(p) : "r"(x), "n"(BYTES), "l"(base));
  return reinterpret_cast<const uint8_t *>(p);
}

// Warps per CTA, CTAs per SM and chunks in a warp's ring: as many warps as the
// registers of their O (32 per n-tile and d = 128) allow, their rings sharing
// the SM's shared memory.
constexpr int NW = 4;
__host__ __device__ constexpr int ctas_per_sm(bool fp8, int d, int nr) {
  return nr > 2 ? 2 : fp8 ? (nr > 1 ? (d > 64 ? 2 : 3) : 4) : d > 64 ? 2 : 4;
}
__host__ __device__ constexpr int ring_chunks(bool fp8, int d, int nr) {
  return nr > 2 ? (fp8 ? 6 : d > 64 ? 3 : 4) : 3;
}

template <int DH_, bool FP8_, int NR_>
struct Cfg {
  static constexpr int DH = DH_, NR = NR_;
  static constexpr bool FP8 = FP8_;
  static constexpr int CH = chunk_tokens(FP8, NR), MTL = CH / 16;  // tokens of a chunk, their m-tiles
  static constexpr uint32_t ALL = 0xffffffffu >> (32 - CH);
  static constexpr int RB = DH * (FP8 ? 1 : 2);  // bytes per row
  static constexpr int CPR = RB / 16;            // 16-byte pieces per row
  static constexpr int KT = DH / 16;             // k-tiles of S, m-tiles of O
  static constexpr int STAGE = 2 * CH * RB + (FP8 ? 2 * CH * 4 : 0);  // keys, values, their scales
  static constexpr int CTAS = ctas_per_sm(FP8, DH, NR), STAGES = ring_chunks(FP8, DH, NR);
  static constexpr int THREADS = NW * 32;
  static constexpr int R = 8 * NR;
  static constexpr int OROW = DH + 8;  // floats between rows of a warp's result
  static constexpr size_t RING = (size_t)NW * STAGES * STAGE;
  // results of the warps, and of the CTA
  static constexpr size_t JOIN = (size_t)NW * R * (OROW * 4 + 8) + (size_t)R * (DH * 4 + 8);
  static constexpr size_t SMEM = RING > JOIN ? RING : JOIN;
};

// Piece `c` of row `r`: keys are read as 16-byte pieces of two neighbouring
// rows per quarter warp, values by ldmatrix over 8 rows; both without bank
// conflicts under these permutations (each its own inverse).
template <int RB>
__device__ __forceinline__ int k_piece(int r, int c) {
  return RB >= 128 ? c ^ ((r & 1) << 2) : c;
}
template <int RB>
__device__ __forceinline__ int v_piece(int r, int c) {
  return RB >= 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
}

// blockIdx.x: a query (LIST), or a tile of up to `per` queries of a sequence.
template <class F, bool LIST>
__global__ void __launch_bounds__(F::THREADS, F::CTAS)
    attend_kernel(KvView c, AttendView a, Split split, int per) {
  grid_dep_sync();
  constexpr int DH = F::DH, NR = F::NR, R = F::R, RB = F::RB, CPR = F::CPR, KT = F::KT, CH = F::CH,
                MTL = F::MTL;
  constexpr uint32_t ALL = F::ALL;
  constexpr bool FP8 = F::FP8;
  constexpr int STAGES = F::STAGES;
  constexpr bool Q_SMEM = NR > (FP8 ? 1 : 2);  // the query fragments do not fit beside O
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(16) uint2 q_s[Q_SMEM ? KT * NR * 32 : 1];  // [k-tile][pair of n-tiles][lane][2]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c4 = lane & 3;
  const int G = a.H / c.H_kv, hk = blockIdx.y, Z = split.Z;
  int tile_i = blockIdx.x;
  Tile t = {tile_i, 1, 0};
  if (!LIST) t = find_tile<F::THREADS>(a, per, tile_i);

  for (; t.n > 0;) {
    const int n_rows = t.n * G;  // at most R
    auto row_query = [&](int r) { return LIST ? t.q0 : t.q0 + r / G; };
    auto row_head = [&](int r) { return hk * G + (LIST ? r : r % G); };

    // ---- the tile's tokens: prefix (or list) chunks, then drafted chunks ----
    int seq = -1, len = 0, cb, ce;
    int c1 = cdiv(a.k, CH);
    int col_len[NR][2];  // this lane's two columns (rows of the tile) of each n-tile
    auto divide = [&]() {
      const int chunks = c1 + (a.draft_start ? cdiv(a.n_draft, CH) : 0), share = cdiv(chunks, Z);
      cb = min((int)blockIdx.z * share, chunks);
      ce = min(cb + share, chunks);
    };
    // This lane's token (lane & (CH - 1)) of a chunk as listed, before it is checked
    // (the list is read ahead of everything else that the kernel waits for).
    auto listed = [&](int ck) -> int {
      const int i = ck * CH + (lane & (CH - 1));
      if (!LIST) return i;
      return ck < ce && i < a.k ? __ldg(a.topk + (int64_t)t.q0 * a.k + i) : -1;
    };
    int tok_q[STAGES];
    auto read_ahead = [&]() {
#pragma unroll
      for (int st = 0; st < STAGES; ++st) tok_q[st] = listed(cb + warp + st * NW);
    };
    if (LIST) {
      divide();
      read_ahead();
      len = attend_prefix(c, a, t.q0, &seq);
    } else {
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = n * 8 + 2 * c4 + x;
          col_len[n][x] = -1;
          if (r < n_rows) {
            int s;
            col_len[n][x] = attend_prefix(c, a, row_query(r), &s);
            seq = max(seq, s);
            len = max(len, col_len[n][x]);
            if (s < 0) col_len[n][x] = -1;
          }
        }
      len = max(len, __shfl_xor_sync(0xffffffffu, len, 1));
      len = max(len, __shfl_xor_sync(0xffffffffu, len, 2));
      seq = max(seq, __shfl_xor_sync(0xffffffffu, seq, 1));
      seq = max(seq, __shfl_xor_sync(0xffffffffu, seq, 2));
      c1 = cdiv(len, CH);
      divide();
      read_ahead();
    }
    const int n_draft = seq >= 0 && a.draft_start ? a.n_draft : 0;  // a query outside the cache sees none
    const int draft0 = n_draft ? a.draft_start[seq] : 0;
    const int words = cdiv(a.n_draft, 32);

    // ---- query fragments, the k dimension permuted so that a lane's 16-byte
    // pieces of a key row feed whole A fragments ----
    uint2 qf[Q_SMEM ? 1 : KT][Q_SMEM ? 1 : NR];
    auto row_piece = [&](int n, int i) {
      const int r = n * 8 + g;
      // e4m3: 16 elements at 64 ch + 16 c4 (pieces 2 ch, 2 ch + 1 of the lane);
      // bf16: 8 at 32 i + 8 c4
      const int d0 = FP8 ? 64 * (i >> 1) + 16 * c4 + 8 * (i & 1) : 32 * i + 8 * c4;
      return r < n_rows ? *reinterpret_cast<const uint4 *>(a.q + ((int64_t)row_query(r) * a.H + row_head(r)) * DH + d0)
                        : make_uint4(0u, 0u, 0u, 0u);
    };
    // of a product, to a base-2 logit: of this lane's columns, and (e4m3) the
    // power of two of the row that it loads
    float mul[NR][2], sc[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      sc[n] = 1.f;
      mul[n][0] = mul[n][1] = a.scale * LOG2E;
      if (!FP8) continue;
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        const uint4 v = row_piece(n, i);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 f = bf16x2_to_float2(w[p]);
          m = finite_max(finite_max(m, f.x), f.y);
        }
      }
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));  // the row's four lanes
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      sc[n] = f16_scale(m);
#pragma unroll
      for (int x = 0; x < 2; ++x) mul[n][x] *= __shfl_sync(0xffffffffu, inverse(sc[n]), (2 * c4 + x) * 4);
    }
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      if (Q_SMEM && n != warp % NR) continue;  // a warp's share (warps beyond NR repeat, harmlessly)
#pragma unroll
      for (int i = 0; i < DH / 32; ++i) {
        const uint4 v = row_piece(n, i);
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        if (FP8) {
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const float2 f = bf16x2_to_float2(w[p]);
            w[p] = f16x2(f.x * sc[n], f.y * sc[n]);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint2 x = make_uint2(w[2 * u], w[2 * u + 1]);
          if (Q_SMEM)
            q_s[(((2 * i + u) * (NR / 2) + n / 2) * 32 + lane) * 2 + (n & 1)] = x;
          else
            qf[2 * i + u][n] = x;
        }
      }
    }
    if (Q_SMEM) __syncthreads();

    float o[KT][NR][4];
    // per column: base-2 reference of O and of the weights' sum, and the sum
    // over this lane's tokens
    float y_ref[NR][2], l_sum[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
#pragma unroll
      for (int j = 0; j < KT; ++j) o[j][n][0] = o[j][n][1] = o[j][n][2] = o[j][n][3] = 0.f;
      y_ref[n][0] = y_ref[n][1] = NOTHING;
      l_sum[n][0] = l_sum[n][1] = 0.f;
    }

    uint8_t *ring = smem + warp * (STAGES * F::STAGE);
    const uint32_t ring_a = smem_addr(ring);
    const uint8_t *kb = c.k + (int64_t)max(seq, 0) * c.L_cap * c.H_kv * RB;
    const uint8_t *vb = c.v + (int64_t)max(seq, 0) * c.L_cap * c.H_kv * RB;
    const int64_t sb = (int64_t)max(seq, 0) * c.L_cap * c.H_kv;

    // Row of that token within its sequence's keys, token * H_kv + head (below
    // 2^25); -1 for none.
    auto row_of = [&](int ck, int tok) -> int {
      if (ck >= ce) return -1;
      if (ck < c1) {
        if (tok < 0 || tok >= len) return -1;
      } else {
        const int j = (ck - c1) * CH + (lane & (CH - 1));
        if (j >= n_draft) return -1;
        if (LIST && !((a.draft_mask[(int64_t)t.q0 * words + (j >> 5)] >> (j & 31)) & 1u)) return -1;
        const int64_t p = (int64_t)draft0 + j;
        if (p < 0 || p >= c.L_cap) {
          if (LIST) flag(c, MISA_DEV_BAD_POSITION);
          return -1;
        }
        tok = (int)p;
      }
      return tok * c.H_kv + hk;
    };
    // Gather a chunk's rows into stage st; returns which tokens are there.
    // The lane takes piece pc of rows q0r, q0r + RPI, ...; a full chunk (the
    // usual one) copies without predicates.
    constexpr int RPI = 32 / CPR;
    const int q0r = lane / CPR, pc = lane % CPR;
    const uint8_t *kl = kb + pc * 16, *vl = vb + pc * 16;
    const uint32_t dk = ring_a + q0r * RB + k_piece<RB>(q0r, pc) * 16, dv = ring_a + CH * RB + q0r * RB;
    const uint32_t v0 = v_piece<RB>(q0r, pc) * 16;
    auto issue = [&](int at, int row) -> uint32_t {
      const uint32_t have = __ballot_sync(0xffffffffu, row >= 0) & ALL;
      auto copy = [&](auto &&put) {
#pragma unroll
        for (int it = 0; it < CH / RPI; ++it) {
          const uint32_t x = __shfl_sync(0xffffffffu, (uint32_t)max(row, 0), it * RPI + q0r);
          // (the bits of it * RPI and of q0r do not meet)
          put(it, dk + at + it * RPI * RB, row_at<RB>(kl, x),
              dv + at + it * RPI * RB + (v0 ^ v_piece<RB>(it * RPI, 0) * 16), row_at<RB>(vl, x));
        }
      };
      static_assert(RPI % 2 == 0, "k_piece's row parity");
      if (have == ALL) {
        copy([&](int, uint32_t ka, const uint8_t *ks, uint32_t va, const uint8_t *vs) {
          cp_async16(ka, ks);
          cp_async16(va, vs);
        });
      } else if (have) {
        copy([&](int it, uint32_t ka, const uint8_t *ks, uint32_t va, const uint8_t *vs) {
          const bool there = (have >> (it * RPI + q0r)) & 1u;
          cp_async16(ka, ks, there);
          cp_async16(va, vs, there);
        });
      }
      if (FP8 && have && lane < CH) {
        cp_async4(ring_a + at + 2 * CH * RB + lane * 4, c.k_scale + sb + max(row, 0), row >= 0);
        cp_async4(ring_a + at + 2 * CH * RB + (CH + lane) * 4, c.v_scale + sb + max(row, 0), row >= 0);
      }
      cp_async_commit();
      return have;
    };

    int nxt = cb + warp;
    uint32_t have_q[STAGES - 1];
#pragma unroll
    for (int st = 0; st < STAGES - 1; ++st) {
      have_q[st] = issue(st * F::STAGE, row_of(nxt, tok_q[st]));
      nxt += NW;
    }
    int tok_n = tok_q[STAGES - 1];  // read one turn before it is used
    int at = 0, put_at = (STAGES - 1) * F::STAGE;  // stage read now, stage written now
    for (int ck = cb + warp; ck < ce; ck += NW) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();  // every lane's copies have landed, and its reads of the stage issued next are done
      const uint32_t have = have_q[0];
#pragma unroll
      for (int st = 0; st < STAGES - 2; ++st) have_q[st] = have_q[st + 1];
      have_q[STAGES - 2] = issue(put_at, row_of(nxt, tok_n));
      nxt += NW;
      tok_n = listed(nxt);
      uint8_t *sk = ring + at, *sv = sk + CH * RB;
      const float *ss = reinterpret_cast<const float *>(sv + CH * RB);
      put_at = at;
      at = at == (STAGES - 1) * F::STAGE ? 0 : at + F::STAGE;
      if (!have) continue;

      // ---- S^T = K Q^T ----
      float s[NR][MTL][4];
#pragma unroll
      for (int n = 0; n < NR; ++n)
#pragma unroll
        for (int m = 0; m < MTL; ++m) s[n][m][0] = s[n][m][1] = s[n][m][2] = s[n][m][3] = 0.f;
#pragma unroll
      for (int ch = 0; ch < RB / 64; ++ch) {
        uint4 A[MTL], B[MTL], q4 = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int m = 0; m < MTL; ++m) {
          A[m] = *reinterpret_cast<const uint4 *>(sk + (16 * m + g) * RB + k_piece<RB>(g, 4 * ch + c4) * 16);
          B[m] = *reinterpret_cast<const uint4 *>(sk + (16 * m + g + 8) * RB + k_piece<RB>(g, 4 * ch + c4) * 16);
        }
#pragma unroll
        for (int u = 0; u < (FP8 ? 4 : 2); ++u) {
          const int kt = ch * (FP8 ? 4 : 2) + u;
          uint32_t af[MTL][4];
#pragma unroll
          for (int m = 0; m < MTL; ++m) {
            const uint32_t wa[4] = {A[m].x, A[m].y, A[m].z, A[m].w}, wb[4] = {B[m].x, B[m].y, B[m].z, B[m].w};
            if (FP8) {
              widen(wa[u], af[m][0], af[m][2]);
              widen(wb[u], af[m][1], af[m][3]);
            } else {
              af[m][0] = wa[2 * (u & 1)], af[m][1] = wb[2 * (u & 1)];
              af[m][2] = wa[2 * (u & 1) + 1], af[m][3] = wb[2 * (u & 1) + 1];
            }
          }
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            uint2 q;
            if (Q_SMEM) {
              if ((n & 1) == 0) q4 = *reinterpret_cast<const uint4 *>(q_s + ((kt * (NR / 2) + n / 2) * 32 + lane) * 2);
              q = n & 1 ? make_uint2(q4.z, q4.w) : make_uint2(q4.x, q4.y);
            } else {
              q = qf[Q_SMEM ? 0 : kt][Q_SMEM ? 0 : n];
            }
#pragma unroll
            for (int m = 0; m < MTL; ++m)
              FP8 ? mma_f16_16816(s[n][m], af[m], q.x, q.y) : mma_bf16_16816(s[n][m], af[m], q.x, q.y);
          }
        }
      }

      // ---- what each column sees of the chunk ----
      uint32_t vis[NR][2];
      bool masked = have != ALL, mixed = false;  // something is not seen; by some row only
      if (!LIST) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t v = have;
            const int r = n * 8 + 2 * c4 + x;
            if (r < n_rows) {
              if (col_len[n][x] < 0) {
                v = 0u;
              } else if (ck < c1) {
                const int nn = col_len[n][x] - ck * CH;
                v &= nn >= CH ? ALL : nn > 0 ? (1u << nn) - 1u : 0u;
              } else {
                const int j0 = (ck - c1) * CH;
                uint32_t m = a.draft_mask[(int64_t)row_query(r) * words + (j0 >> 5)] >> (j0 & 31) & ALL;
                if (a.n_draft - j0 < CH) m &= (1u << (a.n_draft - j0)) - 1u;
                if (m & ~have) flag(c, MISA_DEV_BAD_POSITION);
                v &= m;
              }
            }
            mixed |= v != have;
            vis[n][x] = v;
          }
        mixed = __any_sync(0xffffffffu, mixed);
        masked |= mixed;
      }

      // ---- weights of the tokens g + 8 y for the columns x: p = e^(s - ref)
      // for the sum, w for the values ----
      float ks[2 * MTL], vs[2 * MTL];
#pragma unroll
      for (int y = 0; y < 2 * MTL; ++y) {
        ks[y] = FP8 ? ss[g + 8 * y] : 1.f;
        vs[y] = FP8 ? ss[CH + g + 8 * y] : 1.f;
      }
      float p[NR][4 * MTL], w[NR][4 * MTL], l_new[NR][2];
      auto logit = [&](auto m, float v, int n, int x, int y) {
        return m.value && !(((LIST ? have : vis[n][x]) >> (g + 8 * y)) & 1u) ? NEG_INF : v;
      };
      // A logit as the reference takes it, rounded.  Against an exact product a
      // reference of 2^27 may be off by 2^3 and more: enough to overflow a weight.
      auto rounded = [&](int n, int x, int y) {
        const float v = s[n][y >> 1][2 * (y & 1) + x];
        return __fmul_rn(FP8 ? __fmul_rn(v, ks[y]) : v, mul[n][x]);
      };
      // m: std::true_type where something is masked; again: behind a reference
      // that has just moved
      auto weigh = [&](auto m, auto again) -> bool {
        float top = 0.f;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          l_new[n][0] = l_new[n][1] = 0.f;
          const uint64_t mul_2 = pair(mul[n][0], mul[n][1]), ref_2 = pair(-y_ref[n][0], -y_ref[n][1]);
#pragma unroll
          for (int y = 0; y < 2 * MTL; ++y) {
            const float s0 = s[n][y >> 1][2 * (y & 1)], s1 = s[n][y >> 1][2 * (y & 1) + 1];
            // (a row's factor last: its power of two and the token's scale may pass fp32's range between them)
            const float2 v2 = again.value ? make_float2(rounded(n, 0, y) - y_ref[n][0], rounded(n, 1, y) - y_ref[n][1])
                              : FP8 ? unpair(fma2(mul2(pair(s0, s1), pair(ks[y], ks[y])), mul_2, ref_2))
                                  : make_float2(fmaf(s0, mul[n][0], -y_ref[n][0]), fmaf(s1, mul[n][1], -y_ref[n][1]));
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int e = 2 * y + x;
              const float v = logit(m, x ? v2.y : v2.x, n, x, y);
              p[n][e] = ex2(v);
              w[n][e] = FP8 ? p[n][e] * vs[y] : p[n][e];
              // (rows gathered for others may hold any scale)
              if (FP8 && !LIST && m.value && v == NEG_INF) w[n][e] = 0.f;
              l_new[n][x] += p[n][e];
              top = fmaxf(top, w[n][e]);
            }
          }
          if (FP8 && fmaxf(l_new[n][0], l_new[n][1]) > SUM_MAX) top = 2.f * LAZY<FP8>;
        }
        return __any_sync(0xffffffffu, top > LAZY<FP8>);
      };
      // (the first visible token always comes out above)
      if (masked ? weigh(std::true_type(), std::false_type()) : weigh(std::false_type(), std::false_type())) {
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float my = NEG_INF;
#pragma unroll
            for (int y = 0; y < 2 * MTL; ++y)
              my = fmaxf(my, logit(std::true_type(), reference<FP8>(rounded(n, x, y), vs[y]), n, x, y));
#pragma unroll
            for (int b = 4; b < 32; b <<= 1) my = fmaxf(my, __shfl_xor_sync(0xffffffffu, my, b));
            const float y_new = fmaxf(y_ref[n][x], my);
            const float al = ex2(y_ref[n][x] - y_new);
            l_sum[n][x] *= al;
#pragma unroll
            for (int j = 0; j < KT; ++j) o[j][n][x] *= al, o[j][n][2 + x] *= al;
            y_ref[n][x] = y_new;
          }
        weigh(std::true_type(), std::true_type());
      }
      uint32_t pb[NR][2 * MTL];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        l_sum[n][0] += l_new[n][0], l_sum[n][1] += l_new[n][1];
#pragma unroll
        for (int y = 0; y < 2 * MTL; ++y)
          pb[n][y] = movmatrix_trans(FP8 ? f16x2(w[n][2 * y], w[n][2 * y + 1]) : bf16x2(w[n][2 * y], w[n][2 * y + 1]));
      }

      // ---- values that some rows must not see: a NaN or infinity there would
      // reach them as 0 * NaN.  Such values are taken out of the chunk and
      // added to the rows that do see them ----
      if (!LIST && mixed) {
        for (int e = lane; e < CH * RB / 4; e += 32) {
          uint32_t *word = reinterpret_cast<uint32_t *>(sv) + e;
          const uint32_t cw = *word;
          const bool bad = FP8 ? __vcmpeq4(cw & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0u
                               : (cw & 0x7f80u) == 0x7f80u || (cw & 0x7f800000u) == 0x7f800000u;
          uint32_t who = __ballot_sync(0xffffffffu, bad);
          while (who) {
            const int src = __ffs(who) - 1;
            who &= who - 1;
            const uint32_t bw = __shfl_sync(0xffffffffu, cw, src);
            const int at = (e - lane + src) * 4, r = at / RB, off = at % RB;
            const int d0 = (v_piece<RB>(r, off >> 4) * 16 + (off & 15)) / (FP8 ? 1 : 2);
            for (int b = 0; b < (FP8 ? 4 : 2); ++b) {
              const uint32_t el = FP8 ? (bw >> (8 * b)) & 0xffu : (bw >> (16 * b)) & 0xffffu;
              if (FP8 ? (el & 0x7fu) != 0x7fu : (el & 0x7f80u) != 0x7f80u) continue;
              const float val = FP8 ? __int_as_float(0x7fffffff) : bf16_bits_to_float(el);
              const int jt = (d0 + b) >> 4, dd = (d0 + b) & 15;
              const int gt = FP8 ? dd >> 1 : dd & 7, hi = FP8 ? dd & 1 : dd >> 3;
#pragma unroll
              for (int n = 0; n < NR; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  float wt = w[n][x];  // token r's weight sits with the lanes of row r % 8
#pragma unroll
                  for (int y = 1; y < 2 * MTL; ++y)
                    if (y == r >> 3) wt = w[n][2 * y + x];
                  wt = __shfl_sync(0xffffffffu, wt, (r & 7) * 4 + c4);
                  if (g != gt || !((vis[n][x] >> r) & 1u)) continue;
#pragma unroll
                  for (int j = 0; j < KT; ++j)
                    if (j == jt) (hi ? o[j][n][2 + x] : o[j][n][x]) += wt * val;
                }
            }
          }
          if (bad) {
            if (FP8) {
              *word = cw & ~__vcmpeq4(cw & 0x7f7f7f7fu, 0x7f7f7f7fu);
            } else {
              *word = ((cw & 0x7f80u) == 0x7f80u ? 0u : cw & 0xffffu) |
                      ((cw & 0x7f800000u) == 0x7f800000u ? 0u : cw & 0xffff0000u);
            }
          }
        }
        __syncwarp();
      }

      // ---- O^T += V^T P^T ----
      const int mi = lane >> 3;
      const uint32_t sva = smem_addr(sv);
#pragma unroll
      for (int j = 0; j < CPR / 2; ++j) {
#pragma unroll
        for (int m = 0; m < MTL; ++m) {
          uint32_t r[4];
          const int vr = 16 * m + (FP8 ? mi & 1 : mi >> 1) * 8 + (lane & 7), pc = 2 * j + (FP8 ? mi >> 1 : mi & 1);
          ldmatrix_x4_trans(r, sva + vr * RB + v_piece<RB>(vr, pc) * 16);
          if (FP8) {
            // a register holds elements (2g, 2g + 1) of tokens 2c and 2c + 1:
            // the even elements are rows 0..7 of an m-tile, the odd ones 8..15
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t af[4];
              widen(__byte_perm(r[2 * h], 0, 0x3120), af[0], af[1]);
              widen(__byte_perm(r[2 * h + 1], 0, 0x3120), af[2], af[3]);
#pragma unroll
              for (int n = 0; n < NR; ++n) mma_f16_16816(o[2 * j + h][n], af, pb[n][2 * m], pb[n][2 * m + 1]);
            }
          } else {
#pragma unroll
            for (int n = 0; n < NR; ++n) mma_bf16_16816(o[j][n], r, pb[n][2 * m], pb[n][2 * m + 1]);
          }
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();  // every ring is free: its memory takes the warps' results

    // ---- join the warps ----
    float *so = reinterpret_cast<float *>(smem);                                      // [NW][R][OROW]
    float2 *syl = reinterpret_cast<float2 *>(smem + (size_t)NW * R * F::OROW * 4);  // [NW][R]
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float l = l_sum[n][x];
#pragma unroll
        for (int b = 4; b < 32; b <<= 1) l += __shfl_xor_sync(0xffffffffu, l, b);
        const int r = warp * R + n * 8 + 2 * c4 + x;
        if (g == 0) syl[r] = make_float2(y_ref[n][x], l);
        float *row = so + (size_t)r * F::OROW;
#pragma unroll
        for (int j = 0; j < KT; ++j) {
          if (FP8) {
            *reinterpret_cast<float2 *>(row + 16 * j + 2 * g) = make_float2(o[j][n][x], o[j][n][2 + x]);
          } else {
            row[16 * j + g] = o[j][n][x];
            row[16 * j + 8 + g] = o[j][n][2 + x];
          }
        }
      }
    __syncthreads();
    float *jo = reinterpret_cast<float *>(syl + NW * R);    // [R][DH]: this CTA's share
    float2 *jyl = reinterpret_cast<float2 *>(jo + R * DH);  // [R]
    const bool in_cluster = Z > 1 && split.o == nullptr;
    auto out_row = [&](int r) { return (int64_t)row_query(r) * a.H + row_head(r); };
    for (int e = tid; e < n_rows * (DH / 4); e += F::THREADS) {
      const int r = e / (DH / 4), d0 = (e % (DH / 4)) * 4;
      const Part p = join_parts<NW>(
          NW, [&](int w) { return syl[w * R + r]; },
          [&](int w) { return *reinterpret_cast<const float4 *>(so + ((size_t)w * R + r) * F::OROW + d0); });
      if (Z == 1) {
        store_row(a, p, out_row(r), DH, d0);
      } else {
        const int64_t prow = (int64_t)blockIdx.z * a.n_q * a.H + out_row(r);
        *reinterpret_cast<float4 *>(in_cluster ? jo + r * DH + d0 : split.o + prow * DH + d0) = p.v;
        if (d0 == 0) *(in_cluster ? jyl + r : split.yl + prow) = make_float2(p.Y, p.l);
      }
    }
    if (in_cluster) {
      // the shares' rows, dealt to the cluster's CTAs (rank = share)
      cluster_sync();
      for (int e = blockIdx.z * F::THREADS + tid; e < n_rows * (DH / 4); e += Z * F::THREADS) {
        const int r = e / (DH / 4), d0 = (e % (DH / 4)) * 4;
        const Part p = join_parts<8>(
            Z, [&](int z) { return ld_cluster2(jyl + r, z); }, [&](int z) { return ld_cluster4(jo + r * DH + d0, z); });
        store_row(a, p, out_row(r), DH, d0);
      }
      cluster_sync();  // no CTA overwrites or leaves what another still reads
    }
    tile_i += gridDim.x;
    if (LIST || tile_i >= t.total) break;
    __syncthreads();
    t = find_tile<F::THREADS>(a, per, tile_i);
  }
}

// One block per row: its four quarters join every fourth share, then meet.
template <int DH>
__global__ void __launch_bounds__(DH) attend_combine_kernel(AttendView a, Split split) {
  grid_dep_sync();
  constexpr int LANES = DH / 4;
  __shared__ float2 yl_s[4];
  __shared__ float4 v_s[4][LANES];
  const int64_t row = blockIdx.x, n = (int64_t)a.n_q * a.H;
  const int part = threadIdx.x / LANES, lane = threadIdx.x % LANES;
  const Part p = join_parts<4>(
      (split.Z - part + 3) / 4, [&](int i) { return split.yl[(int64_t)(4 * i + part) * n + row]; },
      [&](int i) {
        return *reinterpret_cast<const float4 *>(split.o + ((int64_t)(4 * i + part) * n + row) * DH + 4 * lane);
      });
  v_s[part][lane] = p.v;
  if (lane == 0) yl_s[part] = make_float2(p.Y, p.l);
  __syncthreads();
  if (part) return;
  store_row(a, join_parts<4>(4, [&](int i) { return yl_s[i]; }, [&](int i) { return v_s[i][lane]; }), row, DH, 4 * lane);
}

struct Plan {
  int nr;        // n-tiles of 8 rows per CTA
  int per;       // queries per tile (1 with lists)
  int tiles, Z;
  bool cluster;  // the Z shares are a cluster
  bool umma;     // tiles of up to 128 rows on tcgen05 (attend_umma.cu)
};

// Rows of a tile: one query's G heads and, without lists, those of its
// sequence's neighbours.  Lengths are on the device: whole prefixes count as
// full caches, and the batch's queries as spread evenly over the sequences (a
// CTA goes on to the tiles beyond the grid where they are not).
//
// More than 16 rows without lists, or 32 with them, go to the tcgen05 kernel.
// Measured on both (us, mma.sync / tcgen05; 8 sequences, 8 key/value heads of
// 128, 4 heads each; more rows are more queries).  Over 16K tokens, bf16 then
// e4m3: 12 rows 88 / 88 and 65 / 138, 16 rows 88 / 89 and 67 / 140, 20 rows 139 /
// 90 and 110 / 140, 32 rows 142 / 91 and 112 / 142.  Over 1000 tokens: 16 rows
// 15.8 / 16.4 and 16.8 / 25.0, 20 rows 19.5 / 16.8 and 19.9 / 25.2.  Lists of 2048
// tokens (2 key/value heads): 16 rows 8.8 / 13.0 and 9.3 / 19.3, 32 rows 12.3 /
// 13.5 and 13.8 / 19.5.  (17 to 32 rows over e4m3 prefixes would be faster as two
// tiles of mma.sync, with up to 16 heads per key/value head; the rule does not
// tell them apart.)
Plan make_plan(const KvView &c, int n_q, int H, int k, int n_draft) {
  Plan p;
  const int G = H / c.H_kv;
  const bool list = k > 0;
  const int seqs = std::max(1, std::min(n_q, c.n_seq)), per_seq = cdiv(std::max(n_q, 1), seqs);
  const int rows = list ? G : G * std::min(per_seq, 128);
  p.umma = rows > (list ? 32 : 16);
  if (p.umma) {
    p.nr = 0, p.cluster = false;
    p.per = list ? 1 : 128 / G;
    p.tiles = list ? n_q : seqs * cdiv(per_seq, p.per);
    const int chunks = cdiv(list ? k : c.L_cap, 128) + cdiv(n_draft, 128);
    const int64_t units = (int64_t)p.tiles * c.H_kv;
    // shares: the fewest chunk times over the waves of one CTA per SM, with
    // about 8 chunks' time for a CTA's beginning and end
    const int sms = device_sms();
    p.Z = 1;
    int64_t best = INT64_MAX;
    for (int z = 1; z <= std::min(chunks, 32); ++z) {
      const int64_t t = (units * z + sms - 1) / sms * (cdiv(chunks, z) + 8);
      if (t < best) best = t, p.Z = z;
    }
    return p;
  }
  p.nr = rows > 16 ? 4 : rows > 8 ? 2 : 1;
  const int R = 8 * p.nr;
  p.per = list ? 1 : std::max(1, R / G);
  p.tiles = list ? n_q : seqs * cdiv(per_seq, p.per);
  const int ch = chunk_tokens(c.fp8, p.nr), chunks = cdiv(list ? k : c.L_cap, ch) + cdiv(n_draft, ch);
  const int ctas = ctas_per_sm(c.fp8, c.d, p.nr);
  const int64_t units = (int64_t)p.tiles * c.H_kv;
  // shares: fill the SMs once, two chunks per warp at the least.  A cluster of
  // up to 8 joins them without a second launch; more shares pay off only
  // where each of 8 would still run through 32 chunks per warp or more.
  const int64_t want = units > 0 ? (int64_t)device_sms() * ctas / units : 1;
  p.Z = (int)std::max<int64_t>(1, std::min<int64_t>(want, chunks / (2 * NW)));
  if (p.Z > 8 && chunks < 8 * NW * 32) p.Z = 8;
  p.cluster = p.Z > 1 && p.Z <= 8;
  return p;
}

template <class F, bool LIST>
cudaError_t run_attend(const KvView &c, const AttendView &a, const Split &sp, const Plan &p, cudaStream_t s) {
  struct Tag {};
  const int have = cached_per_device<Tag>([] { return opt_in_max_dyn_smem(attend_kernel<F, LIST>); });
  if (have < (int)F::SMEM) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)p.tiles, c.H_kv, p.Z), block(F::THREADS);
  return p.cluster ? launch_kernel_cluster(attend_kernel<F, LIST>, grid, block, dim3(1, 1, p.Z), F::SMEM, s, c, a, sp,
                                           p.per)
                   : launch_kernel(attend_kernel<F, LIST>, grid, block, F::SMEM, s, c, a, sp, p.per);
}

template <int DH, bool FP8, bool LIST>
cudaError_t pick_rows(const KvView &c, const AttendView &a, const Split &sp, const Plan &p, cudaStream_t s) {
  if (p.nr == 1) return run_attend<Cfg<DH, FP8, 1>, LIST>(c, a, sp, p, s);
  if constexpr (LIST)
    if (p.nr == 4) return run_attend<Cfg<DH, FP8, 4>, LIST>(c, a, sp, p, s);
  return run_attend<Cfg<DH, FP8, 2>, LIST>(c, a, sp, p, s);
}

template <int DH, bool FP8>
cudaError_t pick_attend(const KvView &c, const AttendView &a, const Split &sp, const Plan &p, cudaStream_t s) {
  return a.topk ? pick_rows<DH, FP8, true>(c, a, sp, p, s) : pick_rows<DH, FP8, false>(c, a, sp, p, s);
}

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

size_t attend_ws_bytes(const KvView &c, int n_q, int H, int k, int n_draft) {
  const Plan p = make_plan(c, n_q, H, k, n_draft);
  if (p.Z <= 1 || p.cluster) return 0;
  const size_t n = (size_t)p.Z * n_q * H;
  return round256(n * c.d * 4) + round256(n * 8);
}

cudaError_t launch_attend(const KvView &c, const AttendView &a, void *ws, cudaStream_t s) {
  if (a.n_q == 0) return cudaSuccess;
  const Plan p = make_plan(c, a.n_q, a.H, a.topk ? a.k : 0, a.n_draft);
  Split sp = {nullptr, nullptr, p.Z};
  if (p.Z > 1 && !p.cluster) {
    sp.o = static_cast<float *>(ws);
    sp.yl = reinterpret_cast<float2 *>(static_cast<uint8_t *>(ws) + round256((size_t)p.Z * a.n_q * a.H * c.d * 4));
  }
  cudaError_t e = p.umma       ? launch_attend_umma(c, a, sp, p.per, p.tiles, s)
                  : c.d == 128 ? (c.fp8 ? pick_attend<128, true>(c, a, sp, p, s) : pick_attend<128, false>(c, a, sp, p, s))
                             : (c.fp8 ? pick_attend<64, true>(c, a, sp, p, s) : pick_attend<64, false>(c, a, sp, p, s));
  if (e != cudaSuccess || p.Z == 1 || p.cluster) return e;
  const dim3 g((unsigned)(a.n_q * a.H));
  return c.d == 128 ? launch_kernel(attend_combine_kernel<128>, g, dim3(128), 0, s, a, sp)
                    : launch_kernel(attend_combine_kernel<64>, g, dim3(64), 0, s, a, sp);
}

}  // namespace misa
