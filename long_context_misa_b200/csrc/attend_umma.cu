// Attention of tiles with many rows on tcgen05 tensor cores: more than 32
// heads of a query, or of the neighbouring queries of one sequence (drafted
// trees and prefill chunks over whole prefixes).  Same formulas, tokens and
// numbers as attend.cu.
//
// A CTA holds up to 128 rows (lanes of tensor memory) of one key/value head
// and a share of the tokens, in chunks of 64:
//   8 producer warps   gather a chunk's keys (4 warps) and values (4) into
//                      rings of 128-byte-swizzled tiles: cp.async for bf16
//                      rows; e4m3 rows go through a ring of their own and are
//                      widened to f16 by the threads that brought them
//   1 MMA thread       S_j = Q K_j^T and O += P_j V_j (V as the MN-major
//                      operand, P from tensor memory), S_(j+1) before P_j V_j
//   4 softmax warps    one row per thread: S from tensor memory, weights back
//                      into it, the running sum; O is touched only when a
//                      weight passes 256 times its reference
// Tensor memory: O [0, 128), two S of 64 columns, two P of 32.  A tile of 64
// tokens (32 KB bf16) costs 512 cycles of MMA at M = 128 and about 550 of
// softmax issue beside them, against 1425 cycles of its share of HBM.  Tiles
// of 64 tokens keep less of the rings waiting than tiles of 128 (measured:
// see TOK).
#include <type_traits>

#include "attend.cuh"
#include "umma.cuh"

namespace misa {
namespace {

constexpr int M = 128, TOK = 64;  // rows and tokens of a tile
constexpr int W = TOK / 32;        // mask words of a tile
constexpr int WARPS = 13, THREADS = WARPS * 32;
constexpr int PROD0 = 4, MMA_WARP = 12;  // warps 4..7 keys, 8..11 values
constexpr int SLOTS = 32;                // masks and scales in flight (more than the rings can be ahead)
constexpr int T_O = 0, T_S = 128, T_P = 256, T_COLS = 512;
constexpr int BAD = 256;  // non-finite values handled per round

template <int DH_, bool FP8_>
struct UCfg {
  static constexpr int DH = DH_;
  static constexpr bool FP8 = FP8_;
  static constexpr int TILE = TOK * DH * 2;  // one operand tile in shared memory, 16-bit elements
  static constexpr int BLK = TOK * 128;      // its blocks of 64 elements
  static constexpr int QBLK = M * 128, QTILE = M * DH * 2;
  static constexpr int CPR = DH * (FP8 ? 1 : 2) / 16;  // 16-byte pieces of a row as stored
  static constexpr int PER = TOK * CPR / 128;          // of them per producer thread and tile
  static constexpr int RAW = FP8 ? TOK * DH : 0;       // a tile of codes
  // ring stages: operand tiles of keys and values, tiles of codes of either
  static constexpr int NK = FP8 ? 2 : DH > 64 ? 4 : 8, NV = FP8 ? 3 : DH > 64 ? 6 : 10, NR = FP8 ? (DH > 64 ? 5 : 8) : 0;
  static constexpr int SMEM = QTILE + (NK + NV) * TILE + 2 * NR * RAW + 1024;
  static_assert(NV + NR + 2 <= SLOTS, "masks and scales outlive their chunk");
};
constexpr int MAX_STAGES = 10;

struct Shared {
  uint64_t kfull[MAX_STAGES], kempty[MAX_STAGES], vfull[MAX_STAGES], vempty[MAX_STAGES];
  uint64_t sfull[2], sfree[2], pfull[2], pvdone[2], done;
  uint64_t placed[2], scan;  // meetings of a producer group, of the softmax warps
  uint32_t tmem_base;
  int abort;
  int row_idx[2][2][TOK];   // [keys / values][turn][row of the chunk]: row in the sequence, -1 none
  uint32_t have[SLOTS][W];  // which tokens of a chunk are there
  int len[M], query[M];
  int seq, max_len, min_len;
  int n_bad;
  int2 bad_at[BAD];  // (token, element)
  float bad_val[BAD];
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
__global__ void __launch_bounds__(THREADS, 1) attend_umma_kernel(KvView c, AttendView a, Split split, int per) {
  grid_dep_sync();
  constexpr int DH = F::DH, NK = F::NK, NV = F::NV, BLK = F::BLK, TILE = F::TILE, CPR = F::CPR, PER = F::PER;
  constexpr bool FP8 = F::FP8;
  extern __shared__ uint8_t raw_smem[];
  __shared__ Shared sh;
  __shared__ Scales<FP8> scales;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint8_t *smem = raw_smem + ((1024u - (smem_addr(raw_smem) & 1023u)) & 1023u);
  uint8_t *q_s = smem, *k_s = smem + F::QTILE, *v_s = k_s + NK * TILE, *raw_s = v_s + NV * TILE;
  const int G = a.H / c.H_kv, hk = blockIdx.y, Z = split.Z;
  volatile int *abort = &sh.abort;

  int tile_i = blockIdx.x;
  Tile t = {tile_i, 1};
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
        mbar_init(&sh.kfull[i], 128), mbar_init(&sh.vfull[i], FP8 ? 128 : 128 + W);
        mbar_init(&sh.kempty[i], 1), mbar_init(&sh.vempty[i], 1);    // the MMAs' commit
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&sh.sfull[i], 1), mbar_init(&sh.pvdone[i], 1);
        mbar_init(&sh.sfree[i], 128), mbar_init(&sh.pfull[i], 128);  // every softmax thread
      }
      mbar_init(&sh.done, 1);
      mbar_init(&sh.placed[0], 128), mbar_init(&sh.placed[1], 128), mbar_init(&sh.scan, 128);
      fence_mbar_init();
      sh.seq = -1, sh.max_len = 0, sh.min_len = 0x7fffffff;
    }
    __syncthreads();
    if (tid < M) {
      int s = -1, len = 0;
      if (tid < n_rows) {
        len = attend_prefix(c, a, row_query(tid), &s);
        if (s >= 0) {
          sh.seq = s;  // the same in every row that has one
          atomicMax(&sh.max_len, len);
        }
        atomicMin(&sh.min_len, s >= 0 ? len : -1);
      }
      sh.len[tid] = s >= 0 ? len : -1;
      sh.query[tid] = tid < n_rows ? row_query(tid) : -1;
    }
    // ---- Q: 16-bit rows, K-major with 128-byte swizzle; e4m3 caches: f16
    // after a power of two per row ----
    float row_mul = a.scale * LOG2E;
    if (tid < M) {
      const bool live = tid < n_rows;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + ((int64_t)row_query(live ? tid : 0) * a.H + row_head(live ? tid : 0)) * DH);
      float sc = 1.f;
      if (FP8 && live) {
        float m = 0.f;
        for (int p = 0; p < DH / 8; ++p) {
          const uint4 v = src[p];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_float2(w[i]);
            const float x = fabsf(f.x), y = fabsf(f.y);
            m = (x > m || x != x) ? x : m;  // a NaN stays
            m = (y > m || y != y) ? y : m;
          }
        }
        sc = row_scale(m);
        row_mul = a.scale * LOG2E / sc;
      }
      for (int p = 0; p < DH / 8; ++p) {
        uint4 v = live ? src[p] : make_uint4(0u, 0u, 0u, 0u);
        if (FP8) {
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_to_float2(w[i]);
            w[i] = f16x2(f.x * sc, f.y * sc);
          }
          v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4 *>(q_s + tile_at(tid, p, F::QBLK)) = v;
      }
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
      const bool vals = warp >= PROD0 + 4;
      const int pt = (tid - PROD0 * 32) & 127, lt = pt & (TOK - 1);  // (threads beyond TOK repeat the first ones' tokens)
      uint64_t *full = vals ? sh.vfull : sh.kfull, *empty = vals ? sh.vempty : sh.kempty;
      const uint8_t *base = (vals ? c.v : c.k) + (int64_t)max(seq, 0) * c.L_cap * c.H_kv * (CPR * 16);
      const int64_t srow = (int64_t)max(seq, 0) * c.L_cap * c.H_kv;
      uint8_t *ring = vals ? v_s : k_s;
      const int nst = vals ? NV : NK;
      auto listed = [&](int j) -> int {  // token lt of chunk j as listed
        const int i = (cb + j) * TOK + lt;
        if (!LIST) return i;
        return j < n && i < a.k ? __ldg(a.topk + (int64_t)t.q0 * a.k + i) : -1;
      };
      auto row_of = [&](int j, int tok) -> int {
        if (j >= n) return -1;
        if (cb + j < c1) {
          if (tok < 0 || tok >= max_len) return -1;
        } else {
          const int d = (cb + j - c1) * TOK + lt;
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
      // rows of chunk j into row_idx[..][j & 1]; the values' group also notes
      // which are there and (e4m3) brings the scales, for the softmax warps,
      // who wait for the values' tile
      const bool notes = vals && pt < TOK && lane == 0;
      int meetings = 0;
      auto bring_scale = [&](int j, int row) {
        float(*to)[TOK] = pt < TOK ? scales.k : scales.v;
        cp_async4(smem_addr(&to[j & (SLOTS - 1)][lt]), (pt < TOK ? c.k_scale : c.v_scale) + srow + max(row, 0), row >= 0);
      };
      auto place = [&](int j, int row) -> bool {
        if (!LIST && cb + j < c1) {
          const int left = max_len - (cb + j) * TOK - pt;  // (pt is 0 or 32 where it notes)
          if (notes) sh.have[j & (SLOTS - 1)][pt >> 5] = left >= 32 ? 0xffffffffu : left > 0 ? (1u << left) - 1u : 0u;
          if (FP8 && vals) bring_scale(j, row);
          return true;
        }
        if (pt < TOK) sh.row_idx[vals][j & 1][pt] = row;
        const uint32_t b = __ballot_sync(0xffffffffu, row >= 0);
        if (notes) sh.have[j & (SLOTS - 1)][pt >> 5] = b;
        if (FP8 && vals) bring_scale(j, row);
        mbar_arrive(&sh.placed[vals]);
        return wait_bar(&sh.placed[vals], meetings++ & 1, abort, c);
      };
      const int pc = pt % CPR, r0 = pt / CPR;
      constexpr int RSTEP = 128 / CPR;
      // whether chunk j is a stretch of the prefix: its rows need no list, and
      // no meeting of the group to share one
      auto stretch = [&](int j) { return !LIST && cb + j < c1; };
      const uint8_t *lane0 = base + ((int64_t)r0 * c.H_kv + hk) * (CPR * 16) + pc * 16;
      const int64_t step = (int64_t)RSTEP * c.H_kv * (CPR * 16);
      // this thread's pieces of chunk j: rows r0, r0 + RSTEP, ... to at(i, row)
      auto copy = [&](int j, auto &&at) {
        if (stretch(j)) {
          const int t0 = (cb + j) * TOK, left = max_len - t0;
          const uint8_t *p = lane0 + (int64_t)t0 * c.H_kv * (CPR * 16);
          if (left >= TOK) {
#pragma unroll
            for (int i = 0; i < PER; ++i, p += step) cp_async16(at(i, r0 + i * RSTEP), p);
          } else {
#pragma unroll
            for (int i = 0; i < PER; ++i, p += step) {
              const bool there = r0 + i * RSTEP < left;
              cp_async16(at(i, r0 + i * RSTEP), there ? p : base, there);
            }
          }
          return;
        }
        const int *idx = sh.row_idx[vals][j & 1];
#pragma unroll
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
        int tok = listed(0);
        for (int j = 0; j < n; ++j) {
          const int row = row_of(j, tok);
          tok = listed(j + 1);
          if (j >= nst && !wait_bar(&empty[st], wrap, abort, c)) break;
          if (!place(j, row)) break;
          const uint32_t dst = smem_addr(ring + st * TILE);
          copy(j, [&](int, int r) { return dst + tile_at(r, pc, BLK); });
          cp_async_arrive(&full[st]);
          if (notes) mbar_arrive(&full[st]);
          advance();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");  // no copy in flight past here
      } else {
        // codes: NR tiles on their way, each thread its own pieces
        constexpr int NR = F::NR;
        uint8_t *raw = raw_s + (vals ? NR * F::RAW : 0);
        int tok = listed(0);
        auto bring = [&](int j) -> bool {
          const int row = row_of(j, tok);
          tok = listed(j + 1);
          if (j < n) {
            if (!place(j, row)) return false;
            const uint32_t dst = smem_addr(raw + (j % NR) * F::RAW) + pt * 16;
            copy(j, [&](int i, int) { return dst + i * 2048; });
          }
          cp_async_commit();
          return true;
        };
        bool ok = true;
        for (int j = 0; j < NR - 1 && ok; ++j) ok = bring(j);
        for (int j = 0; j < n && ok; ++j) {
          if (!(ok = bring(j + NR - 1))) break;
          cp_async_wait<NR - 1>();
          if (j >= nst && !(ok = wait_bar(&empty[st], wrap, abort, c))) break;
          const uint8_t *from = raw + (j % NR) * F::RAW + pt * 16;
          uint8_t *dst = ring + st * TILE;
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            const uint4 v = *reinterpret_cast<const uint4 *>(from + i * 2048);
            const int r = r0 + i * RSTEP;
            uint32_t w[8];
            widen(v.x, w[0], w[1]), widen(v.y, w[2], w[3]), widen(v.z, w[4], w[5]), widen(v.w, w[6], w[7]);
            *reinterpret_cast<uint4 *>(dst + tile_at(r, 2 * pc, BLK)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4 *>(dst + tile_at(r, 2 * pc + 1, BLK)) = make_uint4(w[4], w[5], w[6], w[7]);
          }
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
        const uint32_t qa = smem_addr(q_s);
        bool ok = true;
        auto pv = [&](int j) {
          const int st = j % NV, b = j & 1;
          ok = ok && wait_bar(&sh.vfull[st], (j / NV) & 1, abort, c) && wait_bar(&sh.pfull[b], (j >> 1) & 1, abort, c);
          if (!ok) return;
          umma::fence_proxy_async();
          umma::fence_after();
          const uint32_t va = smem_addr(v_s + st * TILE);
#pragma unroll
          for (int kk = 0; kk < TOK / 16; ++kk)
            mma_ts(tmem + T_O, tmem + T_P + b * (TOK / 2) + kk * 8, desc_mn(va + kk * 2048, BLK), IDO);
          umma::commit(&sh.vempty[st]);
          umma::commit(&sh.pvdone[b]);
        };
        for (int j = 0; j < n && ok; ++j) {
          const int st = j % NK, b = j & 1;
          ok = wait_bar(&sh.kfull[st], (j / NK) & 1, abort, c) && (j < 2 || wait_bar(&sh.sfree[b], ((j >> 1) & 1) ^ 1, abort, c));
          if (!ok) break;
          umma::fence_proxy_async();
          umma::fence_after();
          const uint32_t ka = smem_addr(k_s + st * TILE);
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) {
            const uint32_t at = (kk & 3) * 32;
            umma::mma<false>(tmem + T_S + b * TOK, umma::smem_desc_sw128(qa + (kk >> 2) * F::QBLK + at),
                             umma::smem_desc_sw128(ka + (kk >> 2) * BLK + at), IDS, kk ? 1u : 0u);
          }
          umma::commit(&sh.kempty[st]);
          umma::commit(&sh.sfull[b]);
          if (j > 0) pv(j - 1);
        }
        if (ok) pv(n - 1);
        // nothing in flight past here (bounded)
        umma::commit(&sh.done);
        mbar_wait(&sh.done, 0);
      }
    } else {
      // ---- softmax: row tid ----
      const uint32_t tl = tmem + ((uint32_t)(warp * 32) << 16);
      const int my_len = sh.len[tid], my_query = sh.query[tid];
      float m_ref = NEG_INF, y_ref = NEG_INF, fac = 1.f, l_sum = 0.f;
      bool ok = true;
      int scans = 0;
      // bounded waits of a whole warp (its tensor-memory accesses need all lanes)
      auto wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait_bar(bar, parity, abort, c)) != 0; };
      auto meet = [&]() {  // the 128 softmax threads
        mbar_arrive(&sh.scan);
        return wait(&sh.scan, scans++ & 1);
      };
      {
        const uint32_t zero[16] = {};
#pragma unroll
        for (int i = 0; i < DH; i += 16) st16(tl + T_O + i, zero);
        st_wait();
      }
      for (int j = 0; j < n && ok; ++j) {
        const int b = j & 1, slot = j & (SLOTS - 1), ck = cb + j;
        ok = wait(&sh.sfull[b], (j >> 1) & 1);
        // P_(j-2) has been used
        if (ok && j >= 2) ok = wait(&sh.pvdone[b], ((j >> 1) & 1) ^ 1);
        // the chunk's masks and scales come with its values (whose stage is
        // not filled again before this chunk is done)
        if (ok) ok = wait(&sh.vfull[j % NV], (j / NV) & 1);
        if (!ok) break;
        umma::fence_after();
        // ---- what this row sees ----
        uint32_t see[W];
        bool masked = false;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t v = sh.have[slot][w];
          if (!LIST) {
            if (ck < c1) {
              const int nn = my_len - ck * TOK - w * 32;
              v &= nn >= 32 ? 0xffffffffu : nn > 0 ? (1u << nn) - 1u : 0u;
            } else if (my_len < 0) {
              v = 0u;
            } else {
              const int d0 = (ck - c1) * TOK + w * 32;
              uint32_t m = d0 < n_draft ? a.draft_mask[(int64_t)my_query * words + (d0 >> 5)] : 0u;
              if (n_draft - d0 < 32) m &= n_draft > d0 ? (1u << (n_draft - d0)) - 1u : 0u;
              if (m & ~v) flag(c, MISA_DEV_BAD_POSITION);
              v &= m;
            }
          }
          if (tid >= n_rows) v = sh.have[slot][w];  // nobody reads these rows
          see[w] = v;
          masked |= v != 0xffffffffu;
        }
        masked = __any_sync(0xffffffffu, masked);
        const uint32_t ts = tl + T_S + b * TOK, tp = tl + T_P + b * (TOK / 2);
        const float *ks = scales.k[FP8 ? slot : 0], *vs = scales.v[FP8 ? slot : 0];

        auto weigh = [&](auto mk, float &sum) -> float {
          float top = 0.f, s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t v[32];
            umma::ld32(ts + w * 32, v);
            umma::ld_wait();
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              float k4[4] = {1.f, 1.f, 1.f, 1.f}, v4[4] = {1.f, 1.f, 1.f, 1.f}, wt[4];
              if (FP8) {
                const float4 x = *reinterpret_cast<const float4 *>(ks + w * 32 + i);
                const float4 y = *reinterpret_cast<const float4 *>(vs + w * 32 + i);
                k4[0] = x.x, k4[1] = x.y, k4[2] = x.z, k4[3] = x.w;
                v4[0] = y.x, v4[1] = y.y, v4[2] = y.z, v4[3] = y.w;
              }
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                float x = fmaf(__uint_as_float(v[i + u]), FP8 ? k4[u] * row_mul : row_mul, -m_ref);
                const bool seen = !mk.value || ((see[w] >> (i + u)) & 1u);
                if (mk.value && !seen) x = NEG_INF;
                const float p = ex2(x);
                s4[u] += p;
                wt[u] = p;
                if (FP8) wt[u] = seen ? p * (v4[u] * fac) : 0.f;
                top = fmaxf(top, fmaxf(p, wt[u]));
              }
#pragma unroll
              for (int u = 0; u < 4; u += 2) pk[(i + u) / 2] = FP8 ? f16x2(wt[u], wt[u + 1]) : bf16x2(wt[u], wt[u + 1]);
            }
            st16(tp + w * 16, pk);
          }
          sum = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          return top;
        };
        float sum = 0.f, top = LAZY + 1.f;
        if (j > 0) top = masked ? weigh(std::true_type(), sum) : weigh(std::false_type(), sum);
        if (__any_sync(0xffffffffu, top > LAZY)) {
          float mx = NEG_INF, my = NEG_INF;
#pragma unroll 1
          for (int w = 0; w < W; ++w) {
            uint32_t v[32];
            umma::ld32(ts + w * 32, v);
            umma::ld_wait();
            const uint32_t sw = w == 0 ? see[0] : see[1];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float x = (sw >> i) & 1u ? __uint_as_float(v[i]) * (FP8 ? ks[w * 32 + i] * row_mul : row_mul) : NEG_INF;
              mx = fmaxf(mx, x);
              if (FP8) {
                const float s = vs[w * 32 + i];
                my = fmaxf(my, x + __log2f(s < 0x1p-100f ? 0x1p-100f : s));  // a NaN stays
              }
            }
          }
          if (!FP8) my = mx;
          const float m_new = fmaxf(m_ref, mx), y_new = fmaxf(y_ref, my);
          l_sum *= m_new == NEG_INF ? 1.f : ex2(m_ref - m_new);
          const float al = y_new == NEG_INF ? 1.f : ex2(y_ref - y_new);
          if (j > 0) {
            // O may change once P_(j-1) V_(j-1) is in it
            ok = wait(&sh.pvdone[b ^ 1], ((j - 1) >> 1) & 1);
            if (!ok) break;
            umma::fence_after();
#pragma unroll 1
            for (int i = 0; i < DH; i += 32) {
              uint32_t v[32];
              umma::ld32(tl + T_O + i, v);
              umma::ld_wait();
              uint32_t x[16], y[16];
#pragma unroll
              for (int u = 0; u < 16; ++u) {
                x[u] = __float_as_uint(__uint_as_float(v[u]) * al);
                y[u] = __float_as_uint(__uint_as_float(v[16 + u]) * al);
              }
              st16(tl + T_O + i, x);
              st16(tl + T_O + i + 16, y);
            }
            st_wait();
          }
          m_ref = m_new, y_ref = y_new;
          fac = m_new == NEG_INF || !FP8 ? 1.f : ex2(m_new - y_new);
          // a row that still sees nothing: its masked logits must not meet -inf
          const float keep = m_ref;
          if (m_ref == NEG_INF) m_ref = 0.f;
          masked ? weigh(std::true_type(), sum) : weigh(std::false_type(), sum);
          m_ref = keep;
        }
        l_sum += sum;
        // ---- values that some rows must not see: NaN and infinities there
        // would reach them as 0 * NaN.  They are taken out of the tile and
        // added to O in the rows that see them (a weight is positive) ----
        if (!LIST && (ck >= c1 || (ck + 1) * TOK > min_len)) {
          if (j > 0) ok = wait(&sh.pvdone[b ^ 1], ((j - 1) >> 1) & 1);
          umma::fence_after();
          uint8_t *vt = v_s + (j % NV) * TILE;
          constexpr uint32_t EXP = FP8 ? 0x7c00u : 0x7f80u;
          int left = 0;
          while (ok) {
            if (!(ok = meet())) break;
            if (tid == 0) sh.n_bad = 0;
            if (!(ok = meet())) break;
            for (int p = 0; p < (tid < TOK ? DH / 8 : 0); ++p) {
              uint16_t *e = reinterpret_cast<uint16_t *>(vt + tile_at(tid, p, BLK));
              const uint4 q = *reinterpret_cast<const uint4 *>(e);
              const uint32_t w[4] = {q.x, q.y, q.z, q.w};
              bool any = false;
#pragma unroll
              for (int i = 0; i < 4; ++i) any |= (w[i] & EXP) == EXP || (w[i] & (EXP << 16)) == EXP << 16;
              if (!any) continue;
              for (int i = 0; i < 8; ++i) {
                const uint32_t bits = e[i];
                if ((bits & EXP) != EXP) continue;
                const int at = atomicAdd(&sh.n_bad, 1);
                if (at >= BAD) continue;  // the next round's
                sh.bad_at[at] = make_int2(tid, p * 8 + i);
                const uint32_t mant = bits & (FP8 ? 0x3ffu : 0x7fu);
                sh.bad_val[at] = mant ? __int_as_float(0x7fffffff) : __int_as_float((bits & 0x8000u) ? 0xff800000u : 0x7f800000u);
                e[i] = 0;
              }
            }
            if (!(ok = meet())) break;
            left = sh.n_bad;
            for (int i = 0; i < min(left, BAD); ++i) {
              const int2 at = sh.bad_at[i];
              const uint32_t sw = at.x < 32 ? see[0] : see[1];
              const uint32_t ov = ld1(tl + T_O + at.y);
              const bool mine = (sw >> (at.x & 31)) & 1u;
              st1(tl + T_O + at.y, mine ? __float_as_uint(__uint_as_float(ov) + sh.bad_val[i]) : ov);
              st_wait();
            }
            if (left <= BAD) break;
          }
          umma::fence_proxy_async();
          if (!ok) break;
        }
        st_wait();
        umma::fence_before();
        mbar_arrive(&sh.sfree[b]);
        mbar_arrive(&sh.pfull[b]);
      }
      if (ok && n > 0) ok = wait(&sh.pvdone[(n - 1) & 1], ((n - 1) >> 1) & 1);
      umma::fence_after();
      // ---- this share of the rows ----
      const bool live = ok && tid < n_rows;
      const int64_t orow = live ? (int64_t)row_query(tid) * a.H + row_head(tid) : 0;
      const int64_t prow = (int64_t)blockIdx.z * a.n_q * a.H + orow;
#pragma unroll 1
      for (int i = 0; i < DH; i += 32) {
        uint32_t v[32];
        umma::ld32(tl + T_O + i, v);
        umma::ld_wait();
        if (!live) continue;
#pragma unroll
        for (int u = 0; u < 32; u += 4) {
          Part p;
          p.M = m_ref, p.Y = y_ref, p.l = l_sum;
          p.v = make_float4(__uint_as_float(v[u]), __uint_as_float(v[u + 1]), __uint_as_float(v[u + 2]), __uint_as_float(v[u + 3]));
          if (Z == 1)
            store_row(a, p, orow, DH, i + u);
          else
            *reinterpret_cast<float4 *>(split.o + prow * DH + i + u) = p.v;
        }
      }
      if (live && Z > 1) split.ml[prow] = make_float4(m_ref, l_sum, y_ref, 0.f);
      umma::fence_before();
    }
    __syncthreads();
    umma::fence_after();
    gave_up = *abort != 0;
    if (LIST || gave_up) break;
    tile_i += gridDim.x;
    t = find_tile<256>(a, per, tile_i);
    if (t.n == 0) break;
    if (tid == 0) {
      for (int i = 0; i < MAX_STAGES; ++i) {
        mbar_inval(&sh.kfull[i]), mbar_inval(&sh.vfull[i]), mbar_inval(&sh.kempty[i]), mbar_inval(&sh.vempty[i]);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_inval(&sh.sfull[i]), mbar_inval(&sh.pvdone[i]), mbar_inval(&sh.sfree[i]), mbar_inval(&sh.pfull[i]);
      }
      mbar_inval(&sh.done), mbar_inval(&sh.placed[0]), mbar_inval(&sh.placed[1]), mbar_inval(&sh.scan);
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
  return launch_kernel(attend_umma_kernel<F, LIST>, dim3((unsigned)tiles, c.H_kv, sp.Z), dim3(THREADS), F::SMEM, s, c, a,
                       sp, per);
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
