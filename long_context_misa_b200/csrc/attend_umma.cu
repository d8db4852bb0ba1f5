// Attention of tiles with many rows on tcgen05 tensor cores: more than 32
// heads of a query with a list, more than 16 of the neighbouring queries of one
// sequence (drafted trees and prefill chunks over whole prefixes).  Same
// formulas, tokens and numbers as attend.cu.
//
// A CTA holds up to 128 rows (lanes of tensor memory) of one key/value head
// and a share of the tokens, in chunks of 128:
//   4 producer warps   bring a chunk's keys (2 warps) and values (2) into
//                      rings of 128-byte-swizzled tiles: TMA for stretches of
//                      a prefix, cp.async for listed and drafted tokens.
//                      e4m3 rows go through a ring of their own and are
//                      widened to f16 there
//   1 MMA thread       S_j = Q K_j^T, a chunk ahead of O += P_j V_j (V as the
//                      MN-major operand, P from tensor memory)
//   2 x 4 softmax warps, one row per thread: a set takes half of a chunk's
//                      tokens, with its own O and running maximum, so that
//                      neither waits for the other; they join at the end.
//                      Weights go back into the columns of S; O is touched
//                      only when a weight has grown more than 256-fold.
// Tensor memory: two O of 128 columns, two S (then P) of 128.
// A chunk (64 KB of bf16 rows) is 1024 cycles of MMA at M = 128 and 2850 of
// the SM's share of HBM.  What decides is the MMA thread: an instruction costs
// it 65 to 85 cycles, a commit or a wait 70, so S is issued at N = 128 for
// both sets (24 queries x 4 heads over 32K bf16 tokens of 4 sequences, 8
// key/value heads: 96 us in bursts, 5.6 TB/s, and 107 in long runs at the card's
// power limit; 143 us with chunks of 64).  128 CTAs are one wave there; a chunk
// takes 1.3 us, the beginning, the end and the join about 15 us.  e4m3 rows have
// half the bytes but take 145 us.  A chunk takes 4200 cycles there, of every
// role: 2200 are a softmax thread's weighing of its 64 tokens (1300 for bf16;
// its exponentials are 1000, two warps on a scheduler's special-function unit),
// the MMA thread waits 1900 for the weights, and what the softmax turn spends
// outside the weighing is not resolved (captured over 8K tokens: issue slots 29 %
// busy; of a warp's stalls per issue 1.7 are short scoreboard, 1.6 instructions
// that have not arrived).  The widening keeps up (eight producer warps, at 96 registers,
// made it 160 us).
#include <type_traits>

#include "attend.cuh"
#include "umma.cuh"

namespace misa {
namespace {

constexpr int M = 128, TOK = 128, HALF = 64;  // rows and tokens of a tile, a set's tokens
constexpr int W = HALF / 32;                  // mask words of a half
constexpr int WARPS = 13, THREADS = WARPS * 32;
constexpr int PROD0 = 8, MMA_WARP = 12;  // warps 0..7 softmax, 8 and 9 keys, 10 and 11 values
constexpr int GROUP = 64;                // threads of a producer group
constexpr int SLOTS = 16;                // masks and scales in flight (more than the rings can be ahead)
constexpr int T_O = 0, T_S = 256, T_COLS = 512;  // O of set g at 128 g, S of chunk j at 256 + 128 (j & 1)
constexpr int BAD = 128;  // non-finite values handled per round

template <int DH_, bool FP8_>
struct UCfg {
  static constexpr int DH = DH_;
  static constexpr bool FP8 = FP8_;
  static constexpr int TILE = TOK * DH * 2;  // one operand tile in shared memory, 16-bit elements
  static constexpr int BLK = TOK * 128;      // its blocks of 64 elements
  static constexpr int QBLK = M * 128, QTILE = M * DH * 2;
  static constexpr int CPR = DH * (FP8 ? 1 : 2) / 16;  // 16-byte pieces of a row as stored
  static constexpr int PER = TOK * CPR / GROUP;        // of them per producer thread and tile
  static constexpr int RAW = FP8 ? TOK * DH : 0;       // a tile of codes
  // ring stages: operand tiles of keys and values, tiles of codes of either
  static constexpr int NK = FP8 ? (DH > 64 ? 1 : 2) : DH > 64 ? 2 : 4, NV = FP8 ? (DH > 64 ? 2 : 3) : DH > 64 ? 3 : 5;
  static constexpr int NR = FP8 ? (DH > 64 ? 2 : 4) : 0;
  static constexpr int SMEM = QTILE + (NK + NV) * TILE + 2 * NR * RAW + 1024;
  static_assert((NK + NV) * TILE >= M * (DH * 4 + 8), "a set's result takes the rings' place");
  static_assert(2 * GROUP == TOK && NV + NR + 2 <= SLOTS, "masks and scales outlive their chunk");
};
constexpr int MAX_STAGES = 5;

struct Shared {
  uint64_t kfull[MAX_STAGES], kempty[MAX_STAGES], vfull[MAX_STAGES], vempty[MAX_STAGES];
  uint64_t rawfull[2][8], rawempty[2][8];
  uint64_t sfull[2], pfull[2][2], pvdone[2], done;  // pfull[set][turn], pvdone[set]
  uint64_t placed[2], scan[2], joined;  // meetings of a producer group, a softmax set, both sets
  uint32_t tmem_base;
  int abort;
  int row_idx[2][2][TOK];   // [keys / values][turn][row of the chunk]: row in the sequence, -1 none
  uint32_t have[SLOTS][2 * W];  // which tokens of a chunk are there
  int len[M], query[M];
  float mul[M];  // of a row's products, to base-2 logits
  int seq, max_len, min_len;
  int n_bad[2];
  int2 bad_at[2][BAD];  // (token, element)
  float bad_val[2][BAD];
};

template <bool FP8>
struct Scales {
  alignas(16) float k[FP8 ? SLOTS : 1][TOK], v[FP8 ? SLOTS : 1][TOK];  // read four at a time
};

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, volatile int *abort, const KvView &c) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    if (globaltimer_ns() - t0 > WAIT_LIMIT_NS) {
      *abort = 1;
      flag(c, MISA_DEV_WAIT_TIMEOUT);
      return false;
    }
  }
  return true;
}

// The same by a whole warp: true in every lane or in none.  A phase may complete
// between two lanes' last polls, and lanes that went on alone would wait for
// ever at the warp's next ballot, vote or tensor-memory access.
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort, const KvView &c) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, c)) != 0;
}

// MN-major, 128-byte swizzle: atoms of 64 elements x 8 k-rows of 128 B; LBO
// steps between 64-element blocks, SBO between groups of 8 k-rows.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t block_bytes) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(block_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, 1, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc));
}

__device__ __forceinline__ void st16(uint32_t t, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t ld1(uint32_t t) {
  uint32_t v;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(t));
  umma::ld_wait();
  return v;
}
__device__ __forceinline__ void st1(uint32_t t, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(t), "r"(v) : "memory");
}

// arrive on `bar` once this thread's copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void mbar_inval(uint64_t *bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// Byte offset of 16-byte piece `pc` (8 elements) of row r in a tile: blocks of
// 64 elements, rows of 128 B, pieces permuted within 8 rows.
__device__ __forceinline__ uint32_t tile_at(int r, int pc, int blk) {
  return (pc >> 3) * blk + r * 128 + (((pc & 7) ^ (r & 7)) << 4);
}

template <class F, bool LIST>
__global__ void __launch_bounds__(THREADS, 1) attend_umma_kernel(KvView c, AttendView a, Split split, int per,
                                                               const __grid_constant__ CUtensorMap kmap,
                                                               const __grid_constant__ CUtensorMap vmap, int tma) {
  grid_dep_sync();
  constexpr int DH = F::DH, NK = F::NK, NV = F::NV, BLK = F::BLK, TILE = F::TILE, CPR = F::CPR, PER = F::PER;
  constexpr bool FP8 = F::FP8;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Shared sh;
  __shared__ Scales<FP8> scales;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t pad = (1024u - (smem_addr(raw_smem) & 1023u)) & 1023u;
  uint32_t dyn;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn));
  if (pad + F::SMEM - 1024 > dyn) {  // a layout and an allocation that disagree
    if (tid == 0) flag(c, MISA_DEV_SMEM_LAYOUT);
    return;
  }
  uint8_t *smem = raw_smem + pad;
  uint8_t *q_s = smem, *k_s = smem + F::QTILE, *v_s = k_s + NK * TILE, *raw_s = v_s + NV * TILE;
  const int G = a.H / c.H_kv, hk = blockIdx.y, Z = split.Z;
  volatile int *abort = &sh.abort;

  int tile_i = blockIdx.x;
  Tile t = {tile_i, 1, 0};
  if (!LIST) t = find_tile<256>(a, per, tile_i);
  if (t.n == 0) return;  // the whole CTA, before anything is allocated

  if (warp == MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sh.tmem_base)),
                 "n"(T_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (tid == 0) sh.abort = 0;

  bool gave_up = false;
  for (;;) {
    const int n_rows = t.n * G;
    auto row_query = [&](int r) { return t.q0 + r / G; };
    auto row_head = [&](int r) { return hk * G + r % G; };
    // ---- barriers, rows ----
    if (tid == 0) {
      for (int i = 0; i < MAX_STAGES; ++i) {
        // every producer thread of the group (bf16: as its copies land, and
        // the lanes that noted the masks)
        mbar_init(&sh.kfull[i], GROUP), mbar_init(&sh.vfull[i], FP8 ? GROUP : GROUP + 2);
        mbar_init(&sh.kempty[i], 1), mbar_init(&sh.vempty[i], 1);  // the MMAs' commit
      }
      for (int i = 0; i < 8; ++i)
        for (int v = 0; v < 2; ++v) mbar_init(&sh.rawfull[v][i], 1), mbar_init(&sh.rawempty[v][i], GROUP);
      for (int i = 0; i < 2; ++i)
        mbar_init(&sh.sfull[i], 1), mbar_init(&sh.pfull[0][i], 128), mbar_init(&sh.pfull[1][i], 128);  // a softmax set
      for (int i = 0; i < 2; ++i)
        mbar_init(&sh.pvdone[i], 1), mbar_init(&sh.placed[i], GROUP), mbar_init(&sh.scan[i], 128);
      mbar_init(&sh.done, 1), mbar_init(&sh.joined, 256);
      fence_mbar_init();
      sh.seq = -1, sh.max_len = 0, sh.min_len = 0x7fffffff;
      sh.n_bad[0] = sh.n_bad[1] = 0;
    }
    __syncthreads();
    if (tid < M) {
      const int r = tid;
      int s = -1, len = 0;
      if (r < n_rows) {
        len = attend_prefix(c, a, row_query(r), &s);
        if (s >= 0) {
          sh.seq = s;  // the same in every row that has one
          atomicMax(&sh.max_len, len);
        }
        atomicMin(&sh.min_len, s >= 0 ? len : -1);
      }
      sh.len[r] = s >= 0 ? len : -1;
      sh.query[r] = r < n_rows ? row_query(r) : -1;
    }
    // ---- Q: 16-bit rows, K-major with 128-byte swizzle; e4m3 caches: f16
    // after a power of two of each row ----
    constexpr int QL = DH / 8, QT = THREADS - M;  // pieces of a row; threads (the others look up the rows meanwhile)
    auto q_piece = [&](int r, int p) {
      return r < n_rows ? reinterpret_cast<const uint4 *>(a.q + ((int64_t)row_query(r) * a.H + row_head(r)) * DH)[p]
                        : make_uint4(0u, 0u, 0u, 0u);
    };
    // (M * QL and QT are whole warps, and the QL lanes of a row are of one)
    for (int e = tid - M; tid >= M && e < M * QL; e += QT) {
      const int r = e / QL, p = e % QL;
      uint4 v = q_piece(r, p);
      if (FP8) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_to_float2(w[i]);
          m = finite_max(finite_max(m, f.x), f.y);
        }
#pragma unroll
        for (int b = 1; b < QL; b <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, b));
        const float sc = f16_scale(m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 f = bf16x2_to_float2(w[i]);
          w[i] = f16x2(f.x * sc, f.y * sc);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
        if (p == 0) sh.mul[r] = a.scale * LOG2E * inverse(sc);
      }
      *reinterpret_cast<uint4 *>(q_s + tile_at(r, p, F::QBLK)) = v;
    }
    umma::fence_proxy_async();
    umma::fence_before();
    __syncthreads();
    umma::fence_after();
    const uint32_t tmem = sh.tmem_base;
    const int seq = sh.seq;
    // ---- the tile's chunks: prefix (or list), then drafted; this CTA's share ----
    const int c1 = seq < 0 ? 0 : cdiv(LIST ? a.k : sh.max_len, TOK);
    const int n_draft = seq >= 0 && a.draft_start ? a.n_draft : 0;
    const int chunks = c1 + cdiv(n_draft, TOK), share = cdiv(chunks, Z), words = cdiv(a.n_draft, 32);
    const int cb = min((int)blockIdx.z * share, chunks), n = min(cb + share, chunks) - cb;
    const int draft0 = n_draft ? a.draft_start[seq] : 0;
    const int max_len = sh.max_len, min_len = sh.min_len;

    if (warp >= PROD0 && warp < MMA_WARP) {
      // ---- producers ----
      const bool vals = warp >= PROD0 + 2;
      const int pt = (tid - PROD0 * 32) & (GROUP - 1);
      uint64_t *full = vals ? sh.vfull : sh.kfull, *empty = vals ? sh.vempty : sh.kempty;
      const uint8_t *base = (vals ? c.v : c.k) + (int64_t)max(seq, 0) * c.L_cap * c.H_kv * (CPR * 16);
      const int64_t srow = (int64_t)max(seq, 0) * c.L_cap * c.H_kv;
      uint8_t *ring = vals ? v_s : k_s;
      const int nst = vals ? NV : NK;
      // this thread's tokens of a chunk: pt and pt + GROUP (h = 0, 1)
      auto listed = [&](int j, int h) -> int {  // as listed
        const int i = (cb + j) * TOK + pt + h * GROUP;
        if (!LIST) return i;
        return j < n && i < a.k ? __ldg(a.topk + (int64_t)t.q0 * a.k + i) : -1;
      };
      auto row_of = [&](int j, int h, int tok) -> int {
        if (j >= n) return -1;
        if (cb + j < c1) {
          if (tok < 0 || tok >= max_len) return -1;
        } else {
          const int d = (cb + j - c1) * TOK + pt + h * GROUP;
          if (d >= n_draft) return -1;
          if (LIST && !((a.draft_mask[(int64_t)t.q0 * words + (d >> 5)] >> (d & 31)) & 1u)) return -1;
          const int64_t p = (int64_t)draft0 + d;
          if (p < 0 || p >= c.L_cap) {
            if (LIST) flag(c, MISA_DEV_BAD_POSITION);
            return -1;
          }
          tok = (int)p;
        }
        return tok * c.H_kv + hk;
      };
      int ahead[2] = {listed(0, 0), listed(0, 1)};  // chunk j's tokens, read a chunk before
      // rows of chunk j into row_idx[..][j & 1]; the values' group also notes
      // which are there and (e4m3) brings the scales, for the softmax warps,
      // who wait for the values' tile
      const bool notes = vals && lane == 0;
      int meetings = 0;
      auto place = [&](int j) -> bool {
        const int rows[2] = {row_of(j, 0, ahead[0]), row_of(j, 1, ahead[1])};
        ahead[0] = listed(j + 1, 0), ahead[1] = listed(j + 1, 1);
        if (FP8 && vals) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int64_t row = srow + max(rows[h], 0);
            cp_async4(smem_addr(&scales.k[j & (SLOTS - 1)][pt + h * GROUP]), c.k_scale + row, rows[h] >= 0);
            cp_async4(smem_addr(&scales.v[j & (SLOTS - 1)][pt + h * GROUP]), c.v_scale + row, rows[h] >= 0);
          }
        }
        if (!LIST && cb + j < c1) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int left = max_len - (cb + j) * TOK - pt - h * GROUP;  // (pt is 0 or 32 where it notes)
            if (notes)
              sh.have[j & (SLOTS - 1)][(pt >> 5) + 2 * h] = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
          }
          return true;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sh.row_idx[vals][j & 1][pt + h * GROUP] = rows[h];
          const uint32_t b = __ballot_sync(0xffffffffu, rows[h] >= 0);
          if (notes) sh.have[j & (SLOTS - 1)][(pt >> 5) + 2 * h] = b;
        }
        mbar_arrive(&sh.placed[vals]);
        return wait_warp(&sh.placed[vals], meetings++ & 1, abort, c);
      };
      const int pc = pt % CPR, r0 = pt / CPR;
      constexpr int RSTEP = GROUP / CPR;
      // whether chunk j is a stretch of the prefix: its rows need no list, and
      // no meeting of the group to share one
      auto stretch = [&](int j) { return !LIST && cb + j < c1; };
      // ... and TMA brings it, what lies behind the prefix included (nobody
      // sees it, and what is not finite there is taken out with the masked)
      auto by_tma = [&](int j) { return tma && stretch(j); };
      const CUtensorMap *map = vals ? &vmap : &kmap;
      const uint8_t *lane0 = base + ((int64_t)r0 * c.H_kv + hk) * (CPR * 16) + pc * 16;
      const int64_t step = (int64_t)RSTEP * c.H_kv * (CPR * 16);
      // this thread's pieces of chunk j: rows r0, r0 + RSTEP, ... to at(i, row)
      auto copy = [&](int j, auto &&at) {
        if (stretch(j)) {
          const int t0 = (cb + j) * TOK, left = max_len - t0;
          const uint8_t *p = lane0 + (int64_t)t0 * c.H_kv * (CPR * 16);
          if (left >= TOK) {
#pragma unroll 8
            for (int i = 0; i < PER; ++i, p += step) cp_async16(at(i, r0 + i * RSTEP), p);
          } else {
#pragma unroll 8
            for (int i = 0; i < PER; ++i, p += step) {
              const bool there = r0 + i * RSTEP < left;
              cp_async16(at(i, r0 + i * RSTEP), there ? p : base, there);
            }
          }
          return;
        }
        const int *idx = sh.row_idx[vals][j & 1];
#pragma unroll 8
        for (int i = 0; i < PER; ++i) {
          const int r = r0 + i * RSTEP, x = idx[r];
          cp_async16(at(i, r), base + (uint64_t)(uint32_t)max(x, 0) * (CPR * 16) + pc * 16, x >= 0);
        }
      };
      int st = 0, wrap = 1;  // ring stage of chunk j, parity of its release
      auto advance = [&]() {
        if (++st == nst) st = 0, wrap ^= 1;
      };
      if (!FP8) {
        for (int j = 0; j < n; ++j) {
          if (j >= nst && !wait_warp(&empty[st], wrap, abort, c)) break;
          if (!place(j)) break;
          const uint32_t dst = smem_addr(ring + st * TILE);
          if (by_tma(j)) {
            if (pt == 0) {
              mbar_arrive_expect_tx(&full[st], TILE);
#pragma unroll
              for (int b = 0; b < DH / 64; ++b)
                umma::tma_load_3d(dst + b * BLK, map, 64 * b, hk, seq * c.L_cap + (cb + j) * TOK, &full[st]);
            } else {
              mbar_arrive(&full[st]);
            }
          } else {
            copy(j, [&](int, int r) { return dst + tile_at(r, pc, BLK); });
            cp_async_arrive(&full[st]);
          }
          if (notes) mbar_arrive(&full[st]);
          advance();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // no copy in flight past here
      } else {
        // codes: NR tiles on their way, each thread its own pieces
        constexpr int NR = F::NR;
        uint8_t *raw = raw_s + (vals ? NR * F::RAW : 0);
        auto bring = [&](int j) -> bool {
          if (j < n) {
            if (!place(j)) return false;
            const uint32_t dst = smem_addr(raw + (j % NR) * F::RAW);
            if (by_tma(j)) {
              // (only pt 0 refills the tile, but its warp goes on or leaves as one)
              if (pt < 32 && j >= NR && !wait_warp(&sh.rawempty[vals][j % NR], ((j / NR) & 1) ^ 1, abort, c)) return false;
              if (pt == 0) {
                mbar_arrive_expect_tx(&sh.rawfull[vals][j % NR], F::RAW);
                umma::tma_load_3d(dst, map, 0, hk, seq * c.L_cap + (cb + j) * TOK, &sh.rawfull[vals][j % NR]);
              }
            } else {
              copy(j, [&](int i, int) { return dst + (i * GROUP + pt) * 16; });
            }
          }
          cp_async_commit();
          return true;
        };
        // the 8 lanes of a row store their even or their odd halves first, so
        // that a store of theirs meets every bank once
        const int odd = (pc * 2) >> 3 & 1;
        bool ok = true;
        for (int j = 0; j < NR - 1 && ok; ++j) ok = bring(j);
        for (int j = 0; j < n && ok; ++j) {
          if (!(ok = bring(j + NR - 1))) break;
          cp_async_wait<NR - 1>();
          if (by_tma(j) && !(ok = wait_warp(&sh.rawfull[vals][j % NR], (j / NR) & 1, abort, c))) break;
          if (j >= nst && !(ok = wait_warp(&empty[st], wrap, abort, c))) break;
          const uint8_t *from = raw + (j % NR) * F::RAW + pt * 16;
          uint8_t *dst = ring + st * TILE;
#pragma unroll 8
          for (int i = 0; i < PER; ++i) {
            const uint4 v = *reinterpret_cast<const uint4 *>(from + i * (GROUP * 16));
            const int r = r0 + i * RSTEP;
            uint32_t w[8];
            widen(odd ? v.z : v.x, w[0], w[1]), widen(odd ? v.w : v.y, w[2], w[3]);
            widen(odd ? v.x : v.z, w[4], w[5]), widen(odd ? v.y : v.w, w[6], w[7]);
            *reinterpret_cast<uint4 *>(dst + tile_at(r, 2 * pc + odd, BLK)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(dst + tile_at(r, 2 * pc + 1 - odd, BLK)) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          mbar_arrive(&sh.rawempty[vals][j % NR]);
          umma::fence_proxy_async();
          mbar_arrive(&full[st]);
          advance();
        }
        cp_async_wait<0>();
      }
    } else if (warp == MMA_WARP) {
      // ---- MMA issuer ----
      if (lane == 0 && n > 0) {
        constexpr uint32_t FMT = FP8 ? 0u : 1u;  // f16 / bf16
        constexpr uint32_t IDS = (1u << 4) | (FMT << 7) | (FMT << 10) | ((uint32_t)(TOK >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
        constexpr uint32_t IDO = (1u << 4) | (FMT << 7) | (FMT << 10) | (1u << 16) | ((uint32_t)(DH >> 3) << 17) |
                                 ((uint32_t)(M >> 4) << 24);
        bool ok = true;
        // Descriptors differ in their low words only (addresses in 16 bytes):
        // the thread's own instructions are the loop's length, so they are
        // kept to an add per product and counters instead of divisions.
        const uint64_t kd0 = umma::smem_desc_sw128(smem_addr(k_s)), qd = umma::smem_desc_sw128(smem_addr(q_s));
        const uint64_t vd0 = desc_mn(smem_addr(v_s), BLK);
        uint32_t kst = 0, kph = 0, vst = 0, vph = 0;
        // rows that cp.async brought become visible to the tensor cores here;
        // TMA's are, and widened ones were made so by who wrote them
        auto fence = [&](int j) {
          if (!FP8 && !(tma && !LIST && cb + j < c1)) umma::fence_proxy_async();
          umma::fence_after();
        };
        auto s_of = [&](int j) {
          // the columns held P_(j-2); set 1's products are the later ones
          if (j >= 2) ok = ok && wait_bar(&sh.pvdone[1], j & 1, abort, c);
          ok = ok && wait_bar(&sh.kfull[kst], kph, abort, c);
          if (!ok) return;
          fence(j);
          const uint64_t kd = kd0 + kst * (TILE >> 4);
          const uint32_t to = tmem + T_S + (j & 1) * TOK;
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
            umma::mma<false>(to, qd + (((kk >> 2) * F::QBLK + (kk & 3) * 32) >> 4),
                             kd + (((kk >> 2) * BLK + (kk & 3) * 32) >> 4), IDS, kk ? 1u : 0u);
          umma::commit(&sh.kempty[kst]);
          umma::commit(&sh.sfull[j & 1]);
          if (++kst == NK) kst = 0, kph ^= 1;
        };
        auto pv = [&](int j) {
          ok = ok && wait_bar(&sh.vfull[vst], vph, abort, c);
          if (!ok) return;
          fence(j);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            ok = ok && wait_bar(&sh.pfull[g][j & 1], (j >> 1) & 1, abort, c);
            if (!ok) return;
            umma::fence_after();
            const uint64_t vd = vd0 + ((vst * TILE + g * HALF * 128) >> 4);
            const uint32_t to = tmem + T_O + g * 128, from = tmem + T_S + (j & 1) * TOK + g * HALF;
#pragma unroll
            for (int kk = 0; kk < HALF / 16; ++kk) mma_ts(to, from + kk * 8, vd + ((kk * 2048) >> 4), IDO);
            umma::commit(&sh.pvdone[g]);
          }
          umma::commit(&sh.vempty[vst]);
          if (++vst == NV) vst = 0, vph ^= 1;
        };
        s_of(0);
        for (int j = 0; j < n && ok; ++j) {
          if (j + 1 < n) s_of(j + 1);
          pv(j);
        }
        // nothing in flight past here (bounded)
        umma::commit(&sh.done);
        mbar_wait(&sh.done, 0);
      }
    } else {
      // ---- softmax: row tid % 128, half g of every chunk ----
      const int g = warp >> 2, r = tid & 127;
      const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16), to = tl + T_O + g * 128;
      const int my_len = sh.len[r], my_query = sh.query[r];
      const float mul = FP8 ? sh.mul[r] : a.scale * LOG2E;
      float y_ref = NOTHING, l_sum = 0.f;  // base-2 reference of O and of the sum, and the sum
      bool ok = true;
      int scans = 0;
      // the row's mask of the first drafted chunk's half, read ahead
      uint32_t drafted[W];
      auto draft_word = [&](int d0) -> uint32_t {
        uint32_t m = !LIST && r < n_rows && my_len >= 0 && d0 < n_draft
                         ? a.draft_mask[(int64_t)my_query * words + (d0 >> 5)]
                         : 0u;
        if (n_draft - d0 < 32) m &= n_draft > d0 ? (1u << (n_draft - d0)) - 1u : 0u;
        return m;
      };
#pragma unroll
      for (int w = 0; w < W; ++w) drafted[w] = draft_word(g * HALF + w * 32);
      auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_warp(bar, parity, abort, c); };
      auto meet = [&]() {  // the 128 threads of the set
        mbar_arrive(&sh.scan[g]);
        return wait(&sh.scan[g], scans++ & 1);
      };
      {
        const uint32_t zero[16] = {};
#pragma unroll
        for (int i = 0; i < DH; i += 16) st16(to + i, zero);
        st_wait();
      }
      for (int j = 0; j < n && ok; ++j) {
        const int slot = j & (SLOTS - 1), ck = cb + j;
        ok = wait(&sh.sfull[j & 1], (j >> 1) & 1);
        // the masks and scales come with the chunk's values (whose stage is
        // not filled again before this chunk is done); a stretch of the prefix
        // needs no mask from there
        const bool stretch = !LIST && ck < c1;
        if (ok && (FP8 || !stretch)) ok = wait(&sh.vfull[j % NV], (j / NV) & 1);
        if (!ok) break;
        umma::fence_after();
        // ---- what this row sees ----
        uint32_t see[W];
        bool masked = false;
        if (stretch) {
          const int left = (r < n_rows ? my_len : max_len) - ck * TOK - g * HALF;
          see[0] = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
          see[1] = left >= 64 ? 0xffffffffu : left > 32 ? (1u << (left - 32)) - 1u : 0u;
          masked = left < HALF;
        } else {
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t v = sh.have[slot][W * g + w];
            if (!LIST && r < n_rows) {  // (nobody reads the other rows)
              const uint32_t m = ck == c1 ? drafted[w] : draft_word((ck - c1) * TOK + g * HALF + w * 32);
              if (m & ~v) flag(c, MISA_DEV_BAD_POSITION);
              v &= m;
            }
            see[w] = v;
            masked |= v != 0xffffffffu;
          }
        }
        masked = __any_sync(0xffffffffu, masked);
        const uint32_t ts = tl + T_S + (j & 1) * TOK + g * HALF;
        const float *ks = scales.k[FP8 ? slot : 0] + g * HALF, *vs = scales.v[FP8 ? slot : 0] + g * HALF;

        uint32_t pk[HALF / 2];  // P as it goes back to tensor memory
        // mk: std::true_type where something is masked; again: behind a
        // reference that has just moved.  Then logits are rounded as it took
        // them: against an exact product a reference of 2^27 may be off by 2^3
        // and more, enough to overflow a weight.
        auto weigh = [&](auto mk, auto again, float &sum) -> float {
          float top = 0.f;
          uint64_t s2[2] = {0u, 0u};  // (pairs of fp32)
          const uint64_t mul_2 = pair(mul, mul), ref_2 = pair(-y_ref, -y_ref);
          uint32_t v[FP8 ? 1 : W][32];
          if (!FP8) {
#pragma unroll
            for (int w = 0; w < W; ++w) umma::ld32(ts + w * 32, v[FP8 ? 0 : w]);
            umma::ld_wait();
          }
#pragma unroll
          for (int w = 0; w < W; ++w) {
            if (FP8) {  // (the scales need the registers)
              umma::ld32(ts + w * 32, v[0]);
              umma::ld_wait();
            }
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float4 k4 = make_float4(1.f, 1.f, 1.f, 1.f), v4 = k4;
              if (FP8) {
                k4 = *reinterpret_cast<const float4 *>(ks + w * 32 + i);
                v4 = *reinterpret_cast<const float4 *>(vs + w * 32 + i);
              }
#pragma unroll
              for (int u = 0; u < 4; u += 2) {
                uint64_t x2 = pair(__uint_as_float(v[FP8 ? 0 : w][i + u]), __uint_as_float(v[FP8 ? 0 : w][i + u + 1]));
                // (the row's factor last: its power of two and a token's scale may pass fp32's range between them)
                if (FP8) x2 = mul2(x2, u ? pair(k4.z, k4.w) : pair(k4.x, k4.y));
                float2 x = unpair(fma2(x2, mul_2, ref_2));
                if (again.value) {  // (one by one: a paired product and its sum come out as one operation)
                  x = unpair(x2);
                  x.x = __fadd_rn(__fmul_rn(x.x, mul), -y_ref), x.y = __fadd_rn(__fmul_rn(x.y, mul), -y_ref);
                }
                const bool seen0 = !mk.value || ((see[w] >> (i + u)) & 1u), seen1 = !mk.value || ((see[w] >> (i + u + 1)) & 1u);
                if (mk.value) x.x = seen0 ? x.x : NEG_INF, x.y = seen1 ? x.y : NEG_INF;
                const float2 p = make_float2(ex2(x.x), ex2(x.y));
                const uint64_t p2 = pair(p.x, p.y);
                s2[u >> 1] = add2(s2[u >> 1], p2);
                float2 wt = p;
                if (FP8) {
                  wt = unpair(mul2(p2, u ? pair(v4.z, v4.w) : pair(v4.x, v4.y)));
                  if (mk.value) wt.x = seen0 ? wt.x : 0.f, wt.y = seen1 ? wt.y : 0.f;
                }
                top = fmaxf(top, fmaxf(wt.x, wt.y));
                pk[(w * 32 + i + u) / 2] = FP8 ? f16x2(wt.x, wt.y) : bf16x2(wt.x, wt.y);
              }
            }
          }
          const float2 s0 = unpair(add2(s2[0], s2[1]));
          sum = s0.x + s0.y;
          return FP8 && sum > SUM_MAX ? 2.f * LAZY<FP8> : top;
        };
        float sum = 0.f, top = 2.f * LAZY<FP8>;
        if (j > 0) top = masked ? weigh(std::true_type(), std::false_type(), sum) : weigh(std::false_type(), std::false_type(), sum);
        if (__any_sync(0xffffffffu, top > LAZY<FP8>)) {
          float my = NEG_INF;
#pragma unroll 1
          for (int w = 0; w < W; ++w) {
            uint32_t v[32];
            umma::ld32(ts + w * 32, v);
            umma::ld_wait();
            const uint32_t sw = w == 0 ? see[0] : see[1];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = __fmul_rn(FP8 ? __fmul_rn(__uint_as_float(v[i]), ks[w * 32 + i]) : __uint_as_float(v[i]), mul);
              if ((sw >> i) & 1u) my = fmaxf(my, reference<FP8>(x, FP8 ? vs[w * 32 + i] : 1.f));
            }
          }
          const float y_new = fmaxf(y_ref, my), al = ex2(y_ref - y_new);
          l_sum *= al;
          if (j > 0) {
            // O may change once P_(j-1) V_(j-1) is in it
            ok = wait(&sh.pvdone[g], (j - 1) & 1);
            if (!ok) break;
            umma::fence_after();
#pragma unroll 1
            for (int i = 0; i < DH; i += 32) {
              uint32_t v[32];
              umma::ld32(to + i, v);
              umma::ld_wait();
              uint32_t x[16], y[16];
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                x[u] = __float_as_uint(__uint_as_float(v[u]) * al);
                y[u] = __float_as_uint(__uint_as_float(v[16 + u]) * al);
              }
              st16(to + i, x);
              st16(to + i + 16, y);
            }
            st_wait();
          }
          y_ref = y_new;
          masked ? weigh(std::true_type(), std::true_type(), sum) : weigh(std::false_type(), std::true_type(), sum);
        }
        l_sum += sum;
#pragma unroll
        for (int i = 0; i < HALF / 2; i += 16) st16(ts + i, reinterpret_cast<const uint32_t(&)[16]>(pk[i]));
        // ---- values that some rows must not see: NaN and infinities there
        // would reach them as 0 * NaN.  What lies behind the longest prefix is
        // cleared; what some rows see is taken out of the tile and added to O
        // in those rows (a weight is positive) ----
        const int first = ck * TOK + g * HALF;  // the half's first token
        if (stretch ? first + HALF > min_len : !LIST) {
          ok = wait(&sh.vfull[j % NV], (j / NV) & 1);
          uint8_t *vt = v_s + (j % NV) * TILE;
          constexpr uint32_t EXP = FP8 ? 0x7c00u : 0x7f80u;
          if (stretch && r < HALF && first + r >= max_len)
            for (int p = 0; p < DH / 8; ++p)
              *reinterpret_cast<uint4 *>(vt + tile_at(g * HALF + r, p, BLK)) = make_uint4(0u, 0u, 0u, 0u);
          // rows of the half that some see and some do not: [r0, r1), their
          // pieces dealt to the set's threads
          const int r0 = stretch ? max(min_len - first, 0) : 0;
          const int r1 = min(stretch ? max_len - first : n_draft - (ck - c1) * TOK - g * HALF, HALF);
          bool some = ok && r0 < r1;  // (the same in the whole set)
          while (some) {
            for (int x = r0 * (DH / 8) + r; x < r1 * (DH / 8); x += 128) {
              const int row = x / (DH / 8), p = x % (DH / 8);
              uint16_t *e = reinterpret_cast<uint16_t *>(vt + tile_at(g * HALF + row, p, BLK));
              const uint4 q = *reinterpret_cast<const uint4 *>(e);
              const uint32_t w[4] = {q.x, q.y, q.z, q.w};
              bool any = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) any |= (w[i] & EXP) == EXP || (w[i] & (EXP << 16)) == EXP << 16;
              if (!any) continue;
              for (int i = 0; i < 8; ++i) {
                const uint32_t bits = e[i];
                if ((bits & EXP) != EXP) continue;
                const int at = atomicAdd(&sh.n_bad[g], 1);
                if (at >= BAD) continue;  // the next round's
                sh.bad_at[g][at] = make_int2(row, p * 8 + i);
                const uint32_t mant = bits & (FP8 ? 0x3ffu : 0x7fu);
                sh.bad_val[g][at] =
                    mant ? __int_as_float(0x7fffffff) : __int_as_float((bits & 0x8000u) ? 0xff800000u : 0x7f800000u);
                e[i] = 0;
              }
            }
            if (!(ok = meet())) break;
            const int found = sh.n_bad[g];
            // the count is read by all before the next scan adds to it: S is a
            // chunk ahead, so a warp may be there while another still reads
            if (found == 0) {
              ok = meet();
              break;
            }
            if (j > 0 && !(ok = wait(&sh.pvdone[g], (j - 1) & 1))) break;  // O may change now
            umma::fence_after();
            for (int i = 0; i < min(found, BAD); ++i) {
              const int2 at = sh.bad_at[g][i];
              const uint32_t sw = at.x < 32 ? see[0] : see[1];
              const uint32_t ov = ld1(to + at.y);
              const bool mine = (sw >> (at.x & 31)) & 1u;
              st1(to + at.y, mine ? __float_as_uint(__uint_as_float(ov) + sh.bad_val[g][i]) : ov);
              st_wait();
            }
            if (!(ok = meet())) break;
            if (r == 0) sh.n_bad[g] = 0;
            if (!(ok = meet())) break;
            some = found > BAD;
          }
          umma::fence_proxy_async();
          if (!ok) break;
        }
        st_wait();
        umma::fence_before();
        mbar_arrive(&sh.pfull[g][j & 1]);
      }
      // ---- the two sets' O meet where the rings were (every tile of them has
      // been used once all products are done) ----
      // (pvdone would not do: a set may be two of its phases behind here, and a
      // parity tells only neighbours apart)
      if (ok && n > 0) ok = wait(&sh.done, 0);
      umma::fence_after();
      float *other = reinterpret_cast<float *>(k_s);                 // [DH / 4][M] float4: thread by thread
      float2 *other_yl = reinterpret_cast<float2 *>(k_s + M * DH * 4);  // [M]
      const bool live = ok && r < n_rows;
      if (g == 1 && ok) {
        other_yl[r] = make_float2(y_ref, l_sum);
#pragma unroll 1
        for (int i = 0; i < DH; i += 32) {
          uint32_t v[32];
          umma::ld32(to + i, v);
          umma::ld_wait();
#pragma unroll
          for (int u = 0; u < 32; u += 4)
            reinterpret_cast<uint4 *>(other)[((i + u) / 4) * M + r] = make_uint4(v[u], v[u + 1], v[u + 2], v[u + 3]);
        }
      }
      mbar_arrive(&sh.joined);
      if (g == 0 && ok && (ok = wait(&sh.joined, 0))) {
        const int64_t orow = live ? (int64_t)row_query(r) * a.H + row_head(r) : 0;
        const int64_t prow = (int64_t)blockIdx.z * a.n_q * a.H + orow;
        const float2 mine = make_float2(y_ref, l_sum), theirs = other_yl[r];
        Part ends;
#pragma unroll 1
        for (int i = 0; i < DH; i += 32) {
          uint32_t v[32];
          umma::ld32(to + i, v);
          umma::ld_wait();
#pragma unroll
          for (int u = 0; u < 32; u += 4) {
            if (!live) break;
            const float4 x = reinterpret_cast<const float4 *>(other)[((i + u) / 4) * M + r];
            const float4 y = make_float4(__uint_as_float(v[u]), __uint_as_float(v[u + 1]), __uint_as_float(v[u + 2]),
                                         __uint_as_float(v[u + 3]));
            ends = join_parts<2>(2, [&](int k) { return k ? theirs : mine; }, [&](int k) { return k ? x : y; });
            if (Z == 1)
              store_row(a, ends, orow, DH, i + u);
            else
              *reinterpret_cast<float4 *>(split.o + prow * DH + i + u) = ends.v;
          }
          __syncwarp();
        }
        if (live && Z > 1) split.yl[prow] = make_float2(ends.Y, ends.l);
      }
      umma::fence_before();
    }
    // what was written to the rings' memory here comes before the next tile's
    // TMA; where a wait ran out, copies may still be on their way: they land
    // well within a millisecond
    umma::fence_proxy_async();
    if (*abort)
      for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000;) {
      }
    __syncthreads();
    umma::fence_after();
    gave_up = *abort != 0;
    tile_i += gridDim.x;
    if (LIST || gave_up || tile_i >= t.total) break;
    t = find_tile<256>(a, per, tile_i);
    if (tid == 0) {
      for (int i = 0; i < MAX_STAGES; ++i)
        mbar_inval(&sh.kfull[i]), mbar_inval(&sh.vfull[i]), mbar_inval(&sh.kempty[i]), mbar_inval(&sh.vempty[i]);
      for (int i = 0; i < 8; ++i)
        for (int v = 0; v < 2; ++v) mbar_inval(&sh.rawfull[v][i]), mbar_inval(&sh.rawempty[v][i]);
      for (int i = 0; i < 2; ++i) mbar_inval(&sh.sfull[i]), mbar_inval(&sh.pfull[0][i]), mbar_inval(&sh.pfull[1][i]);
      for (int i = 0; i < 2; ++i) mbar_inval(&sh.pvdone[i]), mbar_inval(&sh.placed[i]), mbar_inval(&sh.scan[i]);
      mbar_inval(&sh.done), mbar_inval(&sh.joined);
    }
    __syncthreads();
  }
  if (warp == MMA_WARP)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem_base), "n"(T_COLS));
}

template <class F, bool LIST>
cudaError_t run(const KvView &c, const AttendView &a, const Split &sp, int per, int tiles, cudaStream_t s) {
  struct Tag {};
  const int have = cached_per_device<Tag>([] { return opt_in_max_dyn_smem(attend_umma_kernel<F, LIST>); });
  if (have < F::SMEM) return cudaErrorInvalidConfiguration;
  CUtensorMap km = {}, vm = {};
  const unsigned long long tokens = (unsigned long long)c.n_seq * c.L_cap;
  const int tma = !LIST && tokens < 0x7fffff00ull &&
                  umma::make_map_heads(&km, c.k, F::FP8, F::DH, c.H_kv, tokens, F::FP8 ? F::DH : 64, TOK, !F::FP8) &&
                  umma::make_map_heads(&vm, c.v, F::FP8, F::DH, c.H_kv, tokens, F::FP8 ? F::DH : 64, TOK, !F::FP8);
  return launch_kernel(attend_umma_kernel<F, LIST>, dim3((unsigned)tiles, c.H_kv, sp.Z), dim3(THREADS), F::SMEM, s, c, a,
                       sp, per, km, vm, tma);
}

}  // namespace

cudaError_t launch_attend_umma(const KvView &c, const AttendView &a, const Split &sp, int per, int tiles,
                               cudaStream_t s) {
  if (c.d == 128) {
    if (c.fp8)
      return a.topk ? run<UCfg<128, true>, true>(c, a, sp, per, tiles, s) : run<UCfg<128, true>, false>(c, a, sp, per, tiles, s);
    return a.topk ? run<UCfg<128, false>, true>(c, a, sp, per, tiles, s) : run<UCfg<128, false>, false>(c, a, sp, per, tiles, s);
  }
  if (c.fp8)
    return a.topk ? run<UCfg<64, true>, true>(c, a, sp, per, tiles, s) : run<UCfg<64, true>, false>(c, a, sp, per, tiles, s);
  return a.topk ? run<UCfg<64, false>, true>(c, a, sp, per, tiles, s) : run<UCfg<64, false>, false>(c, a, sp, per, tiles, s);
}

}  // namespace misa
