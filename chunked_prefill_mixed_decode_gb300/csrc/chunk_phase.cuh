// The chunk phase of the mixed-batch attention kernels: rows of more than one
// new token on the tcgen05 tensor cores.
#pragma once

#include <cfloat>

#include "attention_step.cuh"
#include "q4.cuh"

namespace {

constexpr int kQSlab = 128 * 128;  // one 128-row x 64-column bf16 slab of a Q tile (128-byte rows)
constexpr int kKVSlab = 64 * 128;  // one 64-key x 64-column bf16 slab of a K or V tile
constexpr int kKeys = kChunkTile;  // keys per KV tile
constexpr int kTilePages = kKeys / kPage;

template <int D>
struct ChCfg {
  static constexpr int NSL = D / 64;                  // 64-column slabs per row
  static constexpr int Q_BYTES = NSL * kQSlab;        // one 128-row Q tile
  static constexpr int Q_OFF = 0;                     // Q tile t at Q_OFF + t * Q_BYTES
  static constexpr int KVS = D == 128 ? 4 : 6;        // K/V pipeline stages
  static constexpr int KV_OFF = 2 * Q_BYTES;          // stage b: K at KV_OFF + b*2*NSL*kKVSlab, V after K
  static constexpr int BAR_OFF = KV_OFF + 2 * KVS * NSL * kKVSlab;
  static constexpr int SMEM = BAR_OFF + 1024;         // dynamic shared memory starts 1024-aligned
  static constexpr int TMEM_COLS = 512;
  static constexpr int O_COL = 128;                   // O of Q tile t at column t * O_COL
  static constexpr int S_COL = 256;                   // S/P buffer b of Q tile t at S_COL + (2t + b) * 64
};

// A work item is a pair of consecutive 128-row Q tiles of one chunk row and KV
// head; both read every K/V tile the pair needs from the same shared stages.
struct ChItem {
  int row, tb, c, hk;
  int n_kt;     // KV tiles the pair needs (those of its later tile)
  int kv0;      // CTA-global index of the item's first KV tile (stage and parity)
  int tok0[2], ntok[2], kv_end[2], nkt[2];  // per Q tile; ntok[1] == 0: no second tile
  int t0[2];    // per Q tile: index of its first KV tile among all tiles its softmax group ran
};

// Part of an item (4-bit pools): of how many it is which, the place of the first,
// and the parity of this one among the parts of each softmax group.  The item's c
// and kv_end then count from the part's first key, and n_kt and nkt are the part's
// own; ns == 1: the whole item.
struct ChPart {
  int ns, part, item0, parity[2];
};

constexpr int kRawStages = 3;  // tiles of 4-bit pages on their way to the dequantizing warps

struct ChBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[8], k_empty[8];  // K stage: free once both S issuers' MMAs are done
  uint64_t v_full[8], v_empty[8];  // V stage: free once the PV issuer's MMAs are done
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];  // [Q tile][S/P buffer]
  uint64_t item_full[2], item_empty[2];
  uint64_t mma_done[3];
  uint64_t part_done[2], part_last[2];  // parts: group t's records are written; whether its part is the last is known
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];  // 4-bit pools: pages as they are stored
  uint32_t tmem;
  int abort;
  ChItem items[2];
  ChPart parts[2];
  int last[2];
  // 4-bit pools: items whose Q tiles have been asked for.  Behind the rest: ahead of
  // `items` it costs a GQA 8B step over bf16 pools 0.6 %.
  int q_asked;
};

static_assert(sizeof(ChBars) <= 1024, "chunk-phase barrier block exceeds its reserved space");
static_assert(ChCfg<128>::SMEM <= 232448 && ChCfg<64>::SMEM <= 232448,
              "chunk phase exceeds the per-CTA shared-memory limit");
static_assert(ChCfg<128>::KVS <= 8 && ChCfg<64>::KVS <= 8, "more K/V stages than barriers");

// Over a 4-bit pool, by one thread once every warp has left the phase: Q tiles that
// a phase given up early still has in flight land, and its barriers, up to `last`,
// are invalidated.  (Here and not at the producer's end, where the loops of the phase
// pay for it in registers: 516 -> 519.6 us, two chunks of 3968 tokens.  The bf16 phase
// keeps no count of its Q tiles: with it a GQA 8B step takes 0.9 % longer, 0.720 ->
// 0.728 ms.  Its waits run for 2 s, a Q tile's copy for a few microseconds.)
__device__ __forceinline__ void close_chunk_barriers(ChBars* bars, uint64_t* last) {
  const int n_q = bars->q_asked;
  if (n_q > 0) mbar_wait(&bars->q_full, (n_q - 1) & 1, nullptr, 200000000ull);
  for (uint64_t* b = &bars->q_full; b <= last; ++b) mbar_inval(b);
}

// wait by lane 0, result and ordering shared with the whole warp
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const volatile int* abort,
                                          uint64_t limit_ns) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, abort, limit_ns) ? 1 : 0;
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __syncwarp();
  return ok != 0;
}

// As warp_wait, the whole warp polling a few times before the clock starts; every
// lane takes the same branch.
__device__ __forceinline__ bool warp_wait_fast(uint64_t* bar, uint32_t parity, const volatile int* abort,
                                               uint64_t limit_ns) {
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, abort, limit_ns);
}

// ---- 4-bit pools: K and V tiles by warps instead of TMA

constexpr int kDequantWarps = kTilePages;            // one per page of a tile
constexpr int kDequantWarp0 = 4 + kSoftmaxWarps;     // warps 12-15

// The phase's shared memory over a 4-bit pool: the bf16 phase's, then the raw pages.
template <int D>
struct ChQ4 {
  static constexpr int RAW_OFF = ChCfg<D>::SMEM;
  static constexpr int RAW_STAGE = kTilePages * Q4<D>::BYTES;
  static constexpr int SMEM = RAW_OFF + kRawStages * RAW_STAGE;
};

// N words of shared memory, 4 N-byte aligned
template <int N>
__device__ __forceinline__ void lds_words(uint32_t src, uint32_t* dst) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(dst[0]), "=r"(dst[1]), "=r"(dst[2]), "=r"(dst[3])
                 : "r"(src)
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(dst[0]), "=r"(dst[1]) : "r"(src) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(dst[0]) : "r"(src) : "memory");
}

// Quarter t of one row (a word per group) as bf16, a quarter of each value, into
// a 128-byte-swizzled tile: group g's eight elements are 16-byte chunk 4 g + t of
// the row, in slab g / 2.
template <int D, int SLAB>
__device__ __forceinline__ void store_row_part(uint32_t row_addr, int key, int t, const uint32_t* words,
                                               const uint32_t* scales) {
  constexpr int NG = Q4<D>::NG;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint32_t s2 = __byte_perm(scales[g >> 1], 0, (g & 1) ? 0x3232 : 0x1010);
    const uint32_t c2 = q4_minus_6(s2);
    uint32_t x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = q4_quarter_pair(words[g], i, s2, c2);
    const uint32_t dst = row_addr + (g >> 1) * SLAB + ((((g & 1) * 4 + t) ^ (key & 7)) << 4);
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                 : "memory");
  }
}

// Warp 12 + w turns page w of every tile into K and V rows of the CTA's items.
// Four lanes share a row (16 bytes of codes each at D = 128); the eight lanes
// of one 16-byte access hold rows r and r ^ 5: they differ in bit 0, so the
// loads cover both halves of a 128-byte line, and in bit 2, so that the stored
// chunks land in different halves of the swizzled line.  Rows past the row's
// context are written as zeros.  Returns false when a wait gave up.
template <int D>
__device__ __forceinline__ bool dequant_role(uint8_t* smem, ChBars* bars, const volatile int* abort_flag, uint64_t lim) {
  using C = ChCfg<D>;
  using Q = Q4<D>;
  constexpr int NSL = C::NSL, NG = Q::NG, KVS = C::KVS;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) - kDequantWarp0;
  const int t = lane & 3, y = lane >> 2;
  const int r0 = (y >> 1) ^ ((y & 1) * 5);  // and r0 + 8
  const uint32_t sbase = smem_u32(smem);
  int bk = 0, br = 0;            // stages of the next tile: K/V and raw
  uint32_t ph = 1, rph = 0;      // their parities: the K/V stage's last release, the raw stage's fill
  for (int n = 0;; ++n) {
    const int slot = n & 1;
    if (!warp_wait(&bars->item_full[slot], (n >> 1) & 1, abort_flag, lim)) return false;
    const ChItem& it = bars->items[slot];  // stable until this role arrives on item_empty
    if (it.row < 0) return true;
    const int n_kt = it.n_kt, kv_max = max(it.kv_end[0], it.kv_end[1]);
    for (int kt = 0; kt < n_kt; ++kt) {
      const int keys = kv_max - kt * kKeys - w * kPage;  // of this page
      uint32_t k[2][NG], v[2][NG], ks[2][NG / 2], vs[2][NG / 2];
      // Each lane waits by itself (a vote after every wait costs 5 % of the rate); one
      // that gave up goes on within the stage's bounds, to the vote at the end of the tile.
      bool ok = mbar_wait_fast(&bars->raw_full[br], rph, abort_flag, 16, lim);
      if (keys > 0) {
        const uint32_t blk = sbase + ChQ4<D>::RAW_OFF + br * ChQ4<D>::RAW_STAGE + w * Q::BYTES;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = r0 + 8 * i;
          lds_words<NG>(blk + r * Q::ROW + t * 4 * NG, k[i]);
          lds_words<NG>(blk + Q::V_OFF + r * Q::ROW + t * 4 * NG, v[i]);
          lds_words<NG / 2>(blk + Q::KS_OFF + r * NG * 2, ks[i]);
          lds_words<NG / 2>(blk + Q::VS_OFF + r * NG * 2, vs[i]);
          if (r >= keys) {  // past the context: scales of zero (the codes are finite whatever they hold)
#pragma unroll
            for (int j = 0; j < NG / 2; ++j) ks[i][j] = vs[i][j] = 0u;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->raw_empty[br]);
      if (++br == kRawStages) {
        br = 0;
        rph ^= 1u;
      }
      // the stage's first round finds both barriers in their initial phase, which counts as released
      ok &= mbar_wait_fast(&bars->v_empty[bk], ph, abort_flag, 16, lim);
      ok &= mbar_wait_fast(&bars->k_empty[bk], ph, abort_flag, 16, lim);
      if (keys > 0) {
        const uint32_t kbase = sbase + C::KV_OFF + bk * 2 * NSL * kKVSlab + w * 2048;
        const uint32_t vbase = sbase + C::KV_OFF + bk * 2 * NSL * kKVSlab + NSL * kKVSlab + w * NSL * 2048;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = r0 + 8 * i;
          store_row_part<D, kKVSlab>(kbase + r * 128, r, t, k[i], ks[i]);
          uint32_t words[NG];  // even elements (first half of the bytes) below odd ones, group by group
#pragma unroll
          for (int g = 0; g < NG; ++g) words[g] = join_halves(v[i][g >> 1], v[i][NG / 2 + (g >> 1)], g & 1);
          store_row_part<D, 2048>(vbase + r * 128, r, t, words, vs[i]);
        }
      }
      fence_proxy_async_smem();
      if (!__all_sync(0xffffffffu, ok)) return false;
      if (lane == 0) {
        mbar_arrive(&bars->k_full[bk]);
        mbar_arrive(&bars->v_full[bk]);
      }
      if (++bk == KVS) {
        bk = 0;
        ph ^= 1u;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->item_empty[slot]);
  }
}

// ---- parts of a chunk item

// The join of a Q tile's parts, at most 32, by the four warps of the group whose
// part was the last.  A warp takes eight rows and two parts at a time, four lanes
// to a row and a quarter of its 16-byte columns to a lane, so that 8 KB (D = 128)
// are asked for at once; a row to a warp waits for each row's records in turn (40 us instead of 7
// for two parts of 128 rows).
template <int D, int G>
__device__ __forceinline__ void merge_parts(const AttnParams& p, const ChItem& it, const ChPart& pt, int t, int w, int lane) {
  constexpr int E = D / 16;  // 16-byte columns to a lane
  const int rows = it.ntok[t] * G, ns = pt.ns, q = lane & 3;
  const ChunkParts cp(p);
  for (int row0 = 8 * w; row0 < rows; row0 += 32) {
    const int row = row0 + (lane >> 2);
    const bool valid = row < rows;
    const int64_t first = static_cast<int64_t>(pt.item0) * p.ch_rec + t * 128 + (valid ? row : row0);
    float M = -FLT_MAX;
#pragma unroll 8
    for (int i = 0; i < ns; ++i) M = fmaxf(M, __ldcg(cp.ml + first + static_cast<int64_t>(i) * p.ch_rec).x);
    float L = 0.f, o[4 * E];
#pragma unroll
    for (int j = 0; j < 4 * E; ++j) o[j] = 0.f;
#pragma unroll 1
    for (int i = 0; i < ns; i += 2) {  // two parts at a time (the last may be alone, and then weighs nothing)
      float2 x[2];
      float4 a[2][E];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t rec = first + static_cast<int64_t>(min(i + h, ns - 1)) * p.ch_rec;
        x[h] = __ldcg(cp.ml + rec);
        const float4* src = reinterpret_cast<const float4*>(cp.acc + rec * D) + q;
#pragma unroll
        for (int j = 0; j < E; ++j) a[h][j] = __ldcg(src + 4 * j);
      }
      if (i + 1 == ns) x[1].y = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (x[h].y == 0.f) continue;  // no key of the row in this part, and no record of sums
        const float wt = ex2(x[h].x - M);
        L += wt * x[h].y;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          o[4 * j] = fmaf(wt, a[h][j].x, o[4 * j]);
          o[4 * j + 1] = fmaf(wt, a[h][j].y, o[4 * j + 1]);
          o[4 * j + 2] = fmaf(wt, a[h][j].z, o[4 * j + 2]);
          o[4 * j + 3] = fmaf(wt, a[h][j].w, o[4 * j + 3]);
        }
      }
    }
    if (valid) {
      const float inv = 4.f / L;  // the records hold quarters
      bf16* dst = p.out + (static_cast<int64_t>(it.tb + it.tok0[t] + row / G) * p.H_q + it.hk * G + row % G) * D;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o[4 * j] * inv, o[4 * j + 1] * inv);
        const __nv_bfloat162 hi = __floats2bfloat162_rn(o[4 * j + 2] * inv, o[4 * j + 3] * inv);
        *reinterpret_cast<uint2*>(dst + 16 * j + 4 * q) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
    }
  }
}

// The end of a part for the four warps of group t: each row's reference maximum
// (log2 units), sum and O as it is in TMEM into the part's records; the last part
// of the item to get here joins them all.  False when a wait gave up.
template <int D, int G>
__device__ __noinline__ bool end_part(const AttnParams& p, ChBars* bars, int slot, int t, float m, float l, uint32_t tO,
                                      const volatile int* abort_flag, uint64_t lim) {
  const ChItem& it = bars->items[slot];
  const ChPart& pt = bars->parts[slot];
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, r = quad * 32 + lane;
  const bool valid = r / G < it.ntok[t];
  const int64_t rec = static_cast<int64_t>(pt.item0 + pt.part) * p.ch_rec + t * 128 + r;
  const ChunkParts cp(p);
  if (valid) cp.ml[rec] = make_float2(m, l);
  if (it.nkt[t] > 0) {
#pragma unroll 1
    for (int cc = 0; cc < D / 32; ++cc) {
      uint32_t rr[32];
      tmem_ld32(tO + cc * 32, rr);
      tmem_wait_ld();
      reg_fence32(rr);
      if (valid) {
        uint4* dst = reinterpret_cast<uint4*>(cp.acc + rec * D + cc * 32);
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = make_uint4(rr[4 * j], rr[4 * j + 1], rr[4 * j + 2], rr[4 * j + 3]);
      }
      __syncwarp();
    }
  }
  __threadfence();  // this part's records are visible before it is counted
  mbar_arrive(&bars->part_done[t]);
  if (quad == 0) {
    if (!warp_wait_fast(&bars->part_done[t], pt.parity[t], abort_flag, lim)) return false;
    if (lane == 0) {
      bars->last[t] = atomicAdd(cp.cnt + 2 * pt.item0 + t, 1) == pt.ns - 1;
      mbar_arrive(&bars->part_last[t]);
    }
  }
  if (!warp_wait_fast(&bars->part_last[t], pt.parity[t], abort_flag, lim)) return false;
  if (bars->last[t]) {
    __threadfence();
    merge_parts<D, G>(p, it, pt, t, quad, lane);
  }
  return true;
}

// Chunk phase.  Warp 0 owns the work queue and streams Q and K/V with TMA (K
// one tile ahead of V); warps 2-5 and 6-9 are two softmax groups, group t
// owning Q tile t of the current pair, one query row per thread over 64-key
// tiles.  The S MMAs of the two groups and the PV MMAs are three independent
// streams, so three warps issue them: warp 1 the S MMAs of group 0, warp 10
// those of group 1, and warp 11 the PV MMAs of both (one issuer would queue
// one group's PV behind the other's S).  Each group has two S buffers in
// TMEM, so its next S is computed while it exponentiates the current one, and
// P (bf16) overwrites the S values it came from, where the PV MMA reads it.
// The two groups run a tile apart at most, so one group's exponentials
// overlap the other group's MMAs.  Returns when the chunk queue is empty; the
// caller owns TMEM and the barrier invalidation.
//
// Over a 4-bit pool (Q4) warp 0 brings the pages of a tile as they are stored,
// one bulk copy a page, into a ring of their own, and four more warps, 12-15,
// write a quarter of their values -- exactly bf16; the score scale and the last
// division make up for the factor -- into the K and V stages: warp 12 + w page w
// of each tile.  Two chunks of 3968 tokens at 0 and 6000, 32 / 8 heads, D = 128:
// 508 us over the same inputs again, 516 to 520 with the inputs changing from call
// to call, 1.25 PFLOP/s, 0.67 of the measured dense rate; the tensor pipe is 55 % and
// the issue slots 59 % busy, so neither is a limit reached.  A tile pair takes about
// 1800 cycles, in which the softmax warps (which spill: 128 registers a thread), the
// dequantizing warps and the issuers are each busy nearly all the time; copies of the
// kernel without any softmax work, or without any dequantizing, took 482 and 487 us
// where the whole took 507.
// Measured and not kept, before the issue by elected lanes (605 us then): loads
// from global memory into the dequantizing warps' registers a tile ahead, without
// the ring (740 us); where items are few, one Q tile for both softmax groups, every
// other K/V tile each (a 512-token chunk alone 58 -> 54 us, beside 64 decodes
// 78 -> 94, and the branches cost the long chunks 4 %).
template <int D, int G, bool Q4 = false>
__device__ __noinline__ void chunk_phase(const CUtensorMap* tm_q_p, const CUtensorMap* tm_k_p,
                                            const CUtensorMap* tm_v_p, const CUtensorMap* tm_vp_p,
                                            const AttnParams& p, uint8_t* smem, uint32_t tmem) {
  using C = ChCfg<D>;
  constexpr int NSL = C::NSL;
  constexpr int TPT = 128 / G;  // query tokens per 128-row Q tile
  constexpr int KVS = C::KVS;
  const CUtensorMap& tm_q = *tm_q_p;
  const CUtensorMap& tm_k = *tm_k_p;
  const CUtensorMap& tm_v = *tm_v_p;
  const CUtensorMap& tm_vp = *tm_vp_p;  // V by whole pages (D = 128)
  ChBars* bars = reinterpret_cast<ChBars*>(smem + C::BAR_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_items = p.hdr[H_NCH_ITEMS];

  const uint32_t sbase = smem_u32(smem);
  auto k_off = [](int b) { return C::KV_OFF + b * 2 * NSL * kKVSlab; };
  auto v_off = [](int b) { return C::KV_OFF + b * 2 * NSL * kKVSlab + NSL * kKVSlab; };
  // A V stage holds its tile page by page: key k of the tile at
  // (k / 16) * kVPage + slab * 2048 + (k % 16) * 128.  A page is one TMA box
  // (two 2 KB boxes of K cost about as much TMA time as one 4 KB box).
  constexpr int kVPage = NSL * 2048;
  auto s_col = [&](int t, int b) { return tmem + C::S_COL + (2 * t + b) * 64; };

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_full, 1);
    mbar_init(&bars->q_empty, 2);  // one commit per S issuer
    for (int b = 0; b < 8; ++b) {  // all of them, so that all can be invalidated
      mbar_init(&bars->k_full[b], Q4 ? kDequantWarps : 1);
      mbar_init(&bars->k_empty[b], 2);
      mbar_init(&bars->v_full[b], Q4 ? kDequantWarps : 1);
      mbar_init(&bars->v_empty[b], 1);
    }
    for (int t = 0; t < 2; ++t)
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars->s_full[t][b], 1);
        mbar_init(&bars->p_full[t][b], 128);  // the four warps of group t
        mbar_init(&bars->o_done[t][b], 1);
      }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->item_full[b], 1);
      // MMA issuers, softmax threads, dequantizing warps
      mbar_init(&bars->item_empty[b], 3 + 32 * kSoftmaxWarps + (Q4 ? kDequantWarps : 0));
    }
    for (int i = 0; i < 3; ++i) mbar_init(&bars->mma_done[i], 1);
    if constexpr (Q4)
      for (int i = 0; i < kRawStages; ++i) {
        mbar_init(&bars->raw_full[i], 1);
        mbar_init(&bars->raw_empty[i], kDequantWarps);
      }
    if constexpr (Q4)
      for (int t = 0; t < 2; ++t) {
        mbar_init(&bars->part_done[t], 128);
        mbar_init(&bars->part_last[t], 1);
      }
    bars->abort = 0;
    if constexpr (Q4) bars->q_asked = 0;
    fence_mbar_init();
  }
  __syncthreads();
  volatile int* abort_flag = &bars->abort;
  const uint64_t lim = p.wait_limit_ns;
  // The MMA issuers.  Over a 4-bit pool a whole warp runs the loop and one elected lane
  // issues, which takes the issue off the critical path: 605 -> 507 us then for chunks of
  // 3968 tokens at 0 and 6000, 32 / 8 heads.  Over a bf16 pool, where the same change
  // measures 522 -> 527 us there and 2060 -> 2110 us beside long decodes (and 69 -> 61 us
  // for D = 64), lane 0 runs it alone.
  auto one = [&] { return !Q4 || elect_one(); };
  auto join = [&] {
    if constexpr (Q4) __syncwarp();
  };
  auto issue_wait = [&](uint64_t* bar, uint32_t parity) {
    return Q4 ? warp_wait_fast(bar, parity, abort_flag, lim) : mbar_wait_fast(bar, parity, abort_flag, 16, lim);
  };
  auto issue_wait_item = [&](uint64_t* bar, uint32_t parity) {
    return Q4 ? warp_wait_fast(bar, parity, abort_flag, lim) : mbar_wait(bar, parity, abort_flag, lim);
  };
  auto softmax_wait = [&](uint64_t* bar, uint32_t parity) {
    return Q4 ? warp_wait_fast(bar, parity, abort_flag, lim) : warp_wait(bar, parity, abort_flag, lim);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- work queue + TMA producer
    // The whole warp runs this loop: lane 0 owns the queue, the waits and the
    // barrier bookkeeping; a tile's K boxes -- one per (page, 64-column slab)
    // -- go out as one warp-wide TMA instruction, lane L taking page L / NSL,
    // slab L % NSL; its V boxes likewise, one per page (lanes with slab 0).
    if (lane == 0) {
      prefetch_tmap(&tm_q);
      if constexpr (!Q4) {
        prefetch_tmap(&tm_k);
        prefetch_tmap(NSL == 2 ? &tm_vp : &tm_v);
      }
    }
    constexpr int kPageBytes = q4_block_bytes(D), kRawOff = ChQ4<D>::RAW_OFF;
    // lane -> (page, slab); over a 4-bit pool a page is one copy
    const int my_pg = Q4 ? lane : lane / NSL, my_s = Q4 ? 0 : lane % NSL;
    const bool loader = lane < kTilePages * (Q4 ? 1 : NSL);
    int g = 0;               // CTA-global KV tile counter
    int g_v = 0;             // tiles whose V has been issued
    int n_done = 0;          // items taken by this CTA
    int t_run[2] = {0, 0};   // KV tiles run by each softmax group so far
    // Test hook (never set by a real call): publish no work item and issue no
    // copy, as a producer that stopped would.  Every other role then waits on
    // an item that never comes until its bounded wait gives up, with nothing
    // in flight: the timeout path runs exactly as it would in a real stall.
    const bool stalled = p.test_stall != 0;
    bool ok = !stalled;
    auto lane0_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
      int r = 1;
      if (lane == 0) r = mbar_wait(bar, parity, abort_flag, lim) ? 1 : 0;
      r = __shfl_sync(0xffffffffu, r, 0);
      return r != 0;
    };
    // V of tile gv (one tile behind K): its stage was last read by the PV MMAs of gv - KVS
    auto load_v = [&](int gv, int row0, int npg) -> bool {
      const int bv = gv % KVS;
      if (gv >= KVS && !lane0_wait(&bars->v_empty[bv], ((gv / KVS) - 1) & 1)) return false;
      if (lane == 0) mbar_arrive_expect_tx(&bars->v_full[bv], npg * kPage * D * 2);
      __syncwarp();
      if constexpr (NSL == 2) {
        if (loader && my_s == 0 && my_pg < npg)
          tma_load_4d(smem + v_off(bv) + my_pg * kVPage, &tm_vp, 0, 0, 0, row0 / kPage, &bars->v_full[bv]);
      } else {
        if (loader && my_pg < npg)
          tma_load_2d(smem + v_off(bv) + my_pg * kVPage, &tm_v, 0, row0, &bars->v_full[bv]);
      }
      return true;
    };
    const int part_tiles = Q4 ? p.hdr[H_CH_TILES] : 0;
    int kt0 = 0;                // the part's first KV tile
    int parts_run[2] = {0, 0};  // parts run by each softmax group so far
    while (ok) {
      int item = 0;
      if (lane == 0) item = atomicAdd(p.hdr + H_CH_CTR, 1);
      item = __shfl_sync(0xffffffffu, item, 0);
      const int slot = n_done & 1;
      if (n_done >= 2 && !lane0_wait(&bars->item_empty[slot], ((n_done >> 1) - 1) & 1)) {
        ok = false;
        break;
      }
      ChItem it;
      ChPart pt{};
      it.row = -1;
      if (item < n_items) {
        // (chunk row index and, above it, the part; KV head << 16 | pair from the last)
        const int2 kl = __ldg((Q4 && part_tiles > 0 ? ChunkParts(p).items : p.ch_items) + item);
        const int k = Q4 ? kl.x & 0xffff : kl.x;
        it.row = __ldg(p.ch_rows + k);
        it.tb = __ldg(p.cu + it.row);
        const int d = __ldg(p.cu + it.row + 1) - it.tb;
        it.c = __ldg(p.q_start + it.row);
        const int n_qt = (d + TPT - 1) / TPT;
        const int n_pair = (n_qt + 1) >> 1;
        // the prologue ordered the row's items (KV head by KV head, or longest pair
        // first); later Q-tile pairs see more keys
        it.hk = kl.y >> 16;
        const int pair = n_pair - 1 - (kl.y & 0xffff);
        it.n_kt = 0;
        for (int t = 0; t < 2; ++t) {
          const int qt = 2 * pair + t;
          const bool has = qt < n_qt;
          it.tok0[t] = has ? qt * TPT : 0;
          it.ntok[t] = has ? min(TPT, d - qt * TPT) : 0;
          it.kv_end[t] = has ? it.c + it.tok0[t] + it.ntok[t] : 0;
          it.nkt[t] = (it.kv_end[t] + kKeys - 1) / kKeys;
          if constexpr (!Q4) {
            it.t0[t] = t_run[t];
            t_run[t] += it.nkt[t];
          }
          it.n_kt = max(it.n_kt, it.nkt[t]);
        }
        if constexpr (Q4) {
          pt.ns = 1;
          kt0 = 0;
          if (part_tiles > 0) {
            const int ns_row = chunk_parts(it.c, d, part_tiles), per = (it.n_kt + ns_row - 1) / ns_row;
            pt.ns = (it.n_kt + per - 1) / per;
            pt.part = kl.x >> 16;
            pt.item0 = item - pt.part;
            if (pt.part >= pt.ns) continue;  // an earlier pair of the row, with fewer tiles
            kt0 = pt.part * per;
            it.c -= kt0 * kKeys;
            it.n_kt = 0;
            for (int t = 0; t < 2; ++t) {
              it.kv_end[t] -= kt0 * kKeys;
              it.nkt[t] = it.kv_end[t] > 0 ? min(per, (it.kv_end[t] + kKeys - 1) / kKeys) : 0;
              it.n_kt = max(it.n_kt, it.nkt[t]);
              pt.parity[t] = parts_run[t] & 1;
              parts_run[t] += pt.ns > 1 && it.ntok[t] > 0;
            }
          }
          for (int t = 0; t < 2; ++t) {
            it.t0[t] = t_run[t];
            t_run[t] += it.nkt[t];
          }
        }
        it.kv0 = g;
      }
      if (lane == 0) {
        bars->items[slot] = it;
        if constexpr (Q4) bars->parts[slot] = pt;
        mbar_arrive(&bars->item_full[slot]);
      }
      ++n_done;
      if (it.row < 0) break;
      // Q tiles: the previous item's S MMAs must be done with them
      if (n_done >= 2 && !lane0_wait(&bars->q_empty, (n_done - 2) & 1)) {
        ok = false;
        break;
      }
      const int nq = it.ntok[1] > 0 ? 2 : 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars->q_full, nq * 128 * D * 2);
        if constexpr (Q4) bars->q_asked = n_done;
      }
      __syncwarp();
      if (lane < nq * NSL) {
        const int t = lane / NSL, s = lane % NSL;
        tma_load_3d(smem + C::Q_OFF + t * C::Q_BYTES + s * kQSlab, &tm_q, s * 64, it.hk * G, it.tb + it.tok0[t],
                    &bars->q_full);
      }
      const int kv_max = max(it.kv_end[0], it.kv_end[1]);
      const int32_t* btrow = row_table(p, it.row) + (Q4 ? kt0 * kTilePages : 0);
      const int n_pages = (kv_max + kPage - 1) / kPage;
      // lane L < 4 holds the page id of page L of the current tile; the next tile's is in flight
      int pg_cur = lane < kTilePages && lane < n_pages ? __ldg(btrow + lane) : 0;
      int row0_prev = 0, npg_prev = 0;
      for (int kt = 0; kt < it.n_kt; ++kt, ++g) {
        const int lp = (kt + 1) * kTilePages + lane;
        const int pg_nxt = lane < kTilePages && lp < n_pages ? __ldg(btrow + lp) : 0;
        const int b = g % KVS;
        const int keys = min(kKeys, kv_max - kt * kKeys);
        const int npg = (keys + kPage - 1) / kPage;
        int phys = __shfl_sync(0xffffffffu, pg_cur, my_pg & (kTilePages - 1));
        if (loader && my_pg < npg && (phys < 0 || phys >= p.num_pages)) {
          atomicOr(p.hdr + H_STATUS, MS_STATUS_BAD_PAGE);
          phys = 0;
        }
        if constexpr (Q4) {  // the pages as they are stored, one bulk copy each
          const int br = g % kRawStages;
          if (g >= kRawStages && !lane0_wait(&bars->raw_empty[br], ((g / kRawStages) - 1) & 1)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&bars->raw_full[br], npg * kPageBytes);
          __syncwarp();
          if (lane < npg)
            bulk_g2s(smem + kRawOff + (br * kTilePages + lane) * kPageBytes,
                     p.kv_q4 + (static_cast<int64_t>(phys) * p.H_kv + it.hk) * kPageBytes, kPageBytes,
                     &bars->raw_full[br]);
          pg_cur = pg_nxt;
          continue;
        }
        const int row0 = (phys * p.H_kv + it.hk) * kPage;
        // K of tile g: its stage was last read by the S MMAs of tile g - KVS
        if (g >= KVS && !lane0_wait(&bars->k_empty[b], ((g / KVS) - 1) & 1)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[b], npg * kPage * D * 2);
        __syncwarp();
        if (loader && my_pg < npg)
          tma_load_2d(smem + k_off(b) + my_s * kKVSlab + my_pg * 2048, &tm_k, my_s * 64, row0, &bars->k_full[b]);
        if (kt >= 1) {
          if (!load_v(g - 1, row0_prev, npg_prev)) {
            ok = false;
            break;
          }
          g_v = g;
        }
        row0_prev = row0;
        npg_prev = npg;
        pg_cur = pg_nxt;
      }
      if (!ok) break;
      if constexpr (!Q4) {
        if (!load_v(g - 1, row0_prev, npg_prev)) {
          ok = false;
          break;
        }
        g_v = g;
      }
    }
    if (lane == 0) {
      if (!ok && !stalled) *abort_flag = 1;
      // copies still in flight must land before the CTA moves on (Q's: close_chunk_barriers)
      if constexpr (Q4) {
        for (int t = (g > kRawStages ? g - kRawStages : 0); t < g; ++t)
          mbar_wait(&bars->raw_full[t % kRawStages], (t / kRawStages) & 1, nullptr, 200000000ull);
        g = 0;  // none straight into the K and V stages
      }
      for (int t = (g > KVS ? g - KVS : 0); t < g; ++t)
        mbar_wait(&bars->k_full[t % KVS], (t / KVS) & 1, nullptr, 200000000ull);
      for (int t = (g_v > KVS ? g_v - KVS : 0); t < g_v; ++t)
        mbar_wait(&bars->v_full[t % KVS], (t / KVS) & 1, nullptr, 200000000ull);
    }
  } else if (warp == 1 || warp == 2 + kSoftmaxWarps) {
    // ---------------------------------------------------------------- S issuer of one group
    // Every S issuer walks every KV tile of the item and commits to the K
    // stage's "empty" barrier (two commits per phase), issuing MMAs only for
    // the tiles its Q tile needs.  It waits for each stage to be full even
    // when it has no MMA for it: that keeps its commits in step with the
    // producer, so a phase can never complete on commits meant for a later one.
    // The issue loops keep every per-item value in registers, step through the
    // stage rings with counters, and build each operand descriptor once per tile:
    // a k-step or a stage only moves the descriptor's start-address field
    // (bytes >> 4, 14 bits, no carry below 256 KB) by a constant.
    const int t = warp == 1 ? 0 : 1;
    if (Q4 || lane == 0) {
      const uint64_t qdesc = smem_desc_sw128(sbase + C::Q_OFF + t * C::Q_BYTES, 16, 1024);
      const uint64_t kdesc0 = smem_desc_sw128(sbase + C::KV_OFF, 16, 1024);
      const uint32_t s_tm = tmem + C::S_COL + 2 * t * 64;
      constexpr uint32_t idesc_full = idesc_bf16_f32(128, kKeys, 0);
      int bk = 0;        // K stage of the next tile
      uint32_t kph = 0;  // its phase parity
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int slot = n & 1;
        if (!issue_wait_item(&bars->item_full[slot], (n >> 1) & 1)) {
          ok = false;
          break;
        }
        const ChItem& it = bars->items[slot];  // stable until this role arrives on item_empty
        const int row = it.row;
        if (row < 0) break;
        const int nkt = it.nkt[t], t0 = it.t0[t], n_kt = it.n_kt;
        const int kv_max = max(it.kv_end[0], it.kv_end[1]);
        if ((Q4 || nkt > 0) && !issue_wait_item(&bars->q_full, n & 1)) {
          ok = false;
          break;
        }
        for (int kt = 0; kt < n_kt; ++kt) {
          if (!issue_wait(&bars->k_full[bk], kph)) {
            ok = false;
            break;
          }
          if (kt < nkt) {
            const int gt = t0 + kt, b = gt & 1;
            // S buffer b last held P of the group's tile gt - 2: its PV MMA must be done
            if (gt >= 2 && !issue_wait(&bars->o_done[t][b], ((gt - 2) >> 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const int keys = kv_max - kt * kKeys;  // at least kKeys but on the last tile
            const uint32_t idesc_s = keys >= kKeys ? idesc_full : idesc_bf16_f32(128, (keys + 15) & ~15, 0);
            const uint64_t kd = kdesc0 + static_cast<uint64_t>((bk * 2 * NSL * kKVSlab) >> 4);
            const uint32_t dcol = s_tm + b * 64;
            if (one()) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint64_t qo = static_cast<uint64_t>(((kk >> 2) * kQSlab + (kk & 3) * 32) >> 4);
                const uint64_t ko = static_cast<uint64_t>(((kk >> 2) * kKVSlab + (kk & 3) * 32) >> 4);
                mma_bf16_ss(dcol, qdesc + qo, kd + ko, idesc_s, kk > 0 ? 1u : 0u);
              }
              mma_commit(&bars->s_full[t][b]);
            }
            join();
          }
          if (one()) {
            mma_commit(&bars->k_empty[bk]);
            if (kt == n_kt - 1) mma_commit(&bars->q_empty);
          }
          join();
          if (++bk == KVS) {
            bk = 0;
            kph ^= 1u;
          }
        }
        if (!ok) break;
        join();
        if (one()) mbar_arrive(&bars->item_empty[slot]);
      }
      if (!ok) *abort_flag = 1;
      // every MMA this thread issued must finish before TMEM is reused or released
      if (one()) {
        mma_commit(&bars->mma_done[t]);
        mbar_wait(&bars->mma_done[t], 0, nullptr, 200000000ull);
      }
    }
  } else if (warp == 3 + kSoftmaxWarps) {
    // ---------------------------------------------------------------- PV issuer of both groups
    if (Q4 || lane == 0) {
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
      // V is the MN-major B operand, one page per k-step of 16 keys: the page's
      // 64-column slabs 2048 B apart (LBO), its two 8-key row groups 1024 B apart
      // (SBO).  P (A operand) is in TMEM: 16 keys = 8 packed columns per k-step.
      const uint64_t vdesc0 = smem_desc_sw128(sbase + C::KV_OFF + NSL * kKVSlab, 2048, 1024);
      int bv = 0;        // V stage of the next tile
      uint32_t vph = 0;  // its phase parity
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int slot = n & 1;
        if (!issue_wait_item(&bars->item_full[slot], (n >> 1) & 1)) {
          ok = false;
          break;
        }
        const ChItem& it = bars->items[slot];  // stable until this role arrives on item_empty
        const int row = it.row;
        if (row < 0) break;
        const int n_kt = it.n_kt;
        const int nkt_[2] = {it.nkt[0], it.nkt[1]}, t0_[2] = {it.t0[0], it.t0[1]};
        const int ke_[2] = {it.kv_end[0], it.kv_end[1]};
        const int kv_max = max(ke_[0], ke_[1]);
        for (int j = 0; j < n_kt && ok; ++j) {
          if (!issue_wait(&bars->v_full[bv], vph)) {
            ok = false;
            break;
          }
          const int keys = min(kKeys, kv_max - j * kKeys);  // keys loaded in this tile
          if (!Q4 && (keys & 15) != 0) {
            // rows past the context in the last page may hold stale (even non-finite)
            // data: zero them in V so that P = 0 times V stays 0
            if (one()) {
              uint8_t* v0 = smem + v_off(bv);
              for (int r = keys; r < ((keys + 15) & ~15); ++r)
                for (int s = 0; s < NSL; ++s)
                  for (int q16 = 0; q16 < 8; ++q16)
                    *reinterpret_cast<uint4*>(v0 + (r >> 4) * kVPage + s * 2048 + (r & 15) * 128 + q16 * 16) =
                        make_uint4(0, 0, 0, 0);
              fence_proxy_async_smem();
            }
            join();
          }
          const uint64_t vd = vdesc0 + static_cast<uint64_t>((bv * 2 * NSL * kKVSlab) >> 4);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (j < nkt_[t]) {
              const int gt = t0_[t] + j, b = gt & 1;
              if (!issue_wait(&bars->p_full[t][b], (gt >> 1) & 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t dcol = tmem + t * C::O_COL;
              const uint32_t acol = s_col(t, b);
              const int kr = ke_[t] - j * kKeys;  // keys this Q tile sees in the tile
              if (one()) {
                if (kr >= kKeys) {
#pragma unroll
                  for (int kk = 0; kk < kKeys / 16; ++kk)
                    mma_bf16_ts(dcol, acol + kk * 8, vd + static_cast<uint64_t>((kk * kVPage) >> 4), idesc_pv,
                                (j > 0 || kk > 0) ? 1u : 0u);
                } else {
                  const int nk_t = (kr + 15) >> 4;
                  for (int kk = 0; kk < nk_t; ++kk)
                    mma_bf16_ts(dcol, acol + kk * 8, vd + static_cast<uint64_t>((kk * kVPage) >> 4), idesc_pv,
                                (j > 0 || kk > 0) ? 1u : 0u);
                }
                mma_commit(&bars->o_done[t][b]);
              }
              join();
            }
          }
          if (!ok) break;
          if (one()) mma_commit(&bars->v_empty[bv]);
          join();
          if (++bv == KVS) {
            bv = 0;
            vph ^= 1u;
          }
        }
        if (!ok) break;
        join();
        if (one()) mbar_arrive(&bars->item_empty[slot]);
      }
      if (!ok) *abort_flag = 1;
      if (one()) {
        mma_commit(&bars->mma_done[2]);
        mbar_wait(&bars->mma_done[2], 0, nullptr, 200000000ull);
      }
    }
  } else if (warp >= 2 && warp < 2 + kSoftmaxWarps) {
    // ---------------------------------------------------------------- softmax
    const int t = (warp - 2) >> 2;              // Q tile of this group
    const int quad = warp & 3;                  // TMEM lane quadrant this warp may access
    const int r = quad * 32 + lane;             // query row of this thread
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tO = tmem + t * C::O_COL + lane_off;
    const float sl2 = Q4 ? 4.f * p.scale_log2 : p.scale_log2;  // Q4: the tiles hold quarters
    // A row exponentiates against m_use, the largest scaled score seen when it
    // was last raised; it is raised (and O rescaled) only when a tile's max
    // exceeds it by more than 2^8, so P <= 256 and O, l stay exact in fp32.
    constexpr float kRescaleLog2 = 8.f;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int slot = n & 1;
      if (!softmax_wait(&bars->item_full[slot], (n >> 1) & 1)) {
        ok = false;
        break;
      }
      const ChItem& it = bars->items[slot];  // stable until this role arrives on item_empty
      if (it.row < 0) break;
      const int nkt = it.nkt[t];
      if (nkt > 0) {
        const int tl = it.tok0[t] + r / G;  // token of this row within the chunk
        const bool valid = (r / G) < it.ntok[t];
        const int pos = it.c + (valid ? tl : it.tok0[t] + it.ntok[t] - 1);
        const int warp_min_pos = it.c + it.tok0[t] + (quad * 32) / G;  // smallest position of this warp's rows
        // (a row may see no key of its part: from the lowest finite number its masked
        // scores have weight 0)
        float m_use = Q4 ? -FLT_MAX : -INFINITY, l = 0.f;
        for (int kt = 0; kt < nkt; ++kt) {
          const int gt = it.t0[t] + kt, b = gt & 1;
          if (!softmax_wait(&bars->s_full[t][b], (gt >> 1) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t r0[32], r1[32];
          const uint32_t ts = s_col(t, b) + lane_off;
          tmem_ld32(ts, r0);
          tmem_ld32(ts + 32, r1);
          tmem_wait_ld();
          reg_fence32(r0);
          reg_fence32(r1);
          float sv[64];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            sv[j] = __uint_as_float(r0[j]);
            sv[32 + j] = __uint_as_float(r1[j]);
          }
          const int key0 = kt * kKeys;
          if (key0 + kKeys - 1 > warp_min_pos) {  // diagonal or ragged tile: causal mask (warp-uniform test)
#pragma unroll
            for (int j = 0; j < 64; ++j)
              if (key0 + j > pos) sv[j] = -INFINITY;
          }
          // row max: four chains of three-input maxima
          float mxa[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            float m = fmax3(sv[c], sv[c + 4], sv[c + 8]);
#pragma unroll
            for (int j = 12; j < 60; j += 8) m = fmax3(m, sv[j + c], sv[j + 4 + c]);
            mxa[c] = fmaxf(m, sv[60 + c]);
          }
          const float mx = fmaxf(fmaxf(mxa[0], mxa[1]), fmaxf(mxa[2], mxa[3]));
          const float mx_s = mx * sl2;
          const bool grow = mx_s > m_use + kRescaleLog2;
          const float m_new = grow ? mx_s : m_use;
          const float alpha = grow ? ex2(m_use - m_new) : 1.f;
          const float neg_m = -m_new;
          // exponentials, two elements per packed FMA and packed add
          const float2 sl2x2 = make_float2(sl2, sl2), negm2 = make_float2(neg_m, neg_m);
          float2 rsa[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int j = 0; j < 64; j += 2) {
            const float2 x = ffma2(make_float2(sv[j], sv[j + 1]), sl2x2, negm2);
            const float2 e = make_float2(ex2(x.x), ex2(x.y));
            sv[j] = e.x;
            sv[j + 1] = e.y;
            rsa[(j >> 1) & 1] = fadd2(rsa[(j >> 1) & 1], e);
          }
          l = l * alpha + ((rsa[0].x + rsa[0].y) + (rsa[1].x + rsa[1].y));
          m_use = m_new;
          // P (bf16 pairs, the operands' type: 2^-9 of each; l is the sum from before) over
          // the first 32 columns of the S values it came from.
          // Packing before the rescale keeps 32 registers live through it instead of
          // 64, and the store runs while O is rescaled.
          uint32_t pw[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            __nv_bfloat162 h2 = __floats2bfloat162_rn(sv[2 * j], sv[2 * j + 1]);
            pw[j] = *reinterpret_cast<uint32_t*>(&h2);
          }
          tmem_st32u(ts, pw);
          if (kt > 0 && __any_sync(0xffffffffu, grow)) {  // rescale this row's O
            // the PV MMA of the previous tile must be done with O first
            if (!softmax_wait(&bars->o_done[t][(gt - 1) & 1], ((gt - 1) >> 1) & 1)) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t rr[32];
              tmem_ld32(tO + cc * 32, rr);
              tmem_wait_ld();
              reg_fence32(rr);
#pragma unroll
              for (int j = 0; j < 32; ++j) rr[j] = __float_as_uint(__uint_as_float(rr[j]) * alpha);
              tmem_st32u(tO + cc * 32, rr);
            }
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(&bars->p_full[t][b]);
        }
        if (!ok) break;
        const int gl = it.t0[t] + nkt - 1;
        if (!softmax_wait(&bars->o_done[t][gl & 1], (gl >> 1) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (Q4 && bars->parts[slot].ns > 1) {
          ok = end_part<D, G>(p, bars, slot, t, m_use, l, tO, abort_flag, lim);
        } else {
          const float inv = (Q4 ? 4.f : 1.f) / l;
          const bool valid_row = Q4 ? r / G < it.ntok[t] : valid;  // read again: a register less in the loop
          bf16* dst = p.out + (static_cast<int64_t>(it.tb + (Q4 ? it.tok0[t] + r / G : tl)) * p.H_q + it.hk * G + r % G) * D;
#pragma unroll
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t rr[32];
            tmem_ld32(tO + cc * 32, rr);
            tmem_wait_ld();
            reg_fence32(rr);
            if (valid_row) {
#pragma unroll
              for (int j = 0; j < 32; j += 8) {
                uint4 u;
                __nv_bfloat162 h0 =
                    __floats2bfloat162_rn(__uint_as_float(rr[j]) * inv, __uint_as_float(rr[j + 1]) * inv);
                __nv_bfloat162 h1 =
                    __floats2bfloat162_rn(__uint_as_float(rr[j + 2]) * inv, __uint_as_float(rr[j + 3]) * inv);
                __nv_bfloat162 h2 =
                    __floats2bfloat162_rn(__uint_as_float(rr[j + 4]) * inv, __uint_as_float(rr[j + 5]) * inv);
                __nv_bfloat162 h3 =
                    __floats2bfloat162_rn(__uint_as_float(rr[j + 6]) * inv, __uint_as_float(rr[j + 7]) * inv);
                u.x = *reinterpret_cast<uint32_t*>(&h0);
                u.y = *reinterpret_cast<uint32_t*>(&h1);
                u.z = *reinterpret_cast<uint32_t*>(&h2);
                u.w = *reinterpret_cast<uint32_t*>(&h3);
                *reinterpret_cast<uint4*>(dst + cc * 32 + j) = u;
              }
            }
          }
        }
      } else if (Q4 && bars->parts[slot].ns > 1 && it.ntok[t] > 0) {  // the part's keys come after all of the tile's tokens
        ok = end_part<D, G>(p, bars, slot, t, -FLT_MAX, 0.f, tO, abort_flag, lim);
      }
      if (Q4 && !ok) break;
      // O has been read: the next item's first PV may overwrite it
      tc_fence_before();
      mbar_arrive(&bars->item_empty[slot]);
    }
    if (!ok) {
      *abort_flag = 1;
      if (lane == 0) atomicOr(p.hdr + H_STATUS, MS_STATUS_TIMEOUT);
    }
  }
  if constexpr (Q4) {
    if (warp >= kDequantWarp0) {
      if (!dequant_role<D>(smem, bars, abort_flag, lim)) *abort_flag = 1;
    }
  }
  (void)n_items;
}

}  // namespace
