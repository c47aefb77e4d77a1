// What every mixed-batch attention kernel starts from: a step's parameters and
// workspace, the one-CTA prologue that validates the rows and lays out the work
// lists, the join of decode splits, and the host side shared by the calls.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "device_state.cuh"
#include "mixed_step.h"
#include "ptx.cuh"

namespace {

using bf16 = __nv_bfloat16;
using namespace ms;

constexpr int kPage = 16;
constexpr int kMinSplitPages = 32;
constexpr int kMaxSplitPages = 256;
constexpr int kSoftmaxWarps = 8;
constexpr int kSortLimit = 2048;    // rows sorted longest-first up to this count
constexpr int kMaxRows = 8192;      // rows of one step
constexpr int kMaxTokens = 1 << 21;  // tokens of one step (a chunk row's Q-tile pairs fit in 16 bits)
// The cost model that splits the SMs between the two row kinds at the start of
// a step needs the SM time of one 128x128 chunk tile and the decode bandwidth
// one SM sustains; both are the attention kernel's own (AttnParams), HBM caps
// the second.
constexpr float kHbmCopyEfficiency = 0.80f;   // sustained share of the nominal HBM rate

// workspace header (int32 words)
enum {
  H_STATUS = 0,
  H_DEC_CTR = 1,
  H_CH_CTR = 2,
  H_NDEC = 3,
  H_NDEC_ITEMS = 4,
  H_NCH = 5,
  H_NCH_ITEMS = 6,
  H_SPLIT = 7,
  H_NPART = 8,
  H_CHUNK_CTAS = 9,  // CTAs that start on chunk work (the rest start on decodes)
  H_CLOCK_MHZ = 10,  // SM clock the last call ran at (kept across calls; 0 in a fresh workspace)
  H_TEAM = 11,       // warps that share a decode item, where the kernel runs them in teams
  H_CH_TILES = 12,   // KV tiles to a part of a chunk item (0: items are whole), where the kernel splits them
  H_WORDS = 64
};

struct AttnParams {
  // Read by the prologue, which runs once per step from cold caches: kept
  // together at the front so that they span the fewest constant-cache lines.
  const int32_t* cu;
  const int32_t* q_start;
  const int32_t* ctx_lens;
  const int32_t* bt_off;  // ragged block table: row s's pages at bt[bt_off[s] .. bt_off[s + 1]); else nullptr
  int32_t* hdr;
  int64_t bt_len;         // entries of bt
  int64_t context_total;
  int64_t max_dec_items, max_ch_items;  // capacities in items (entries x H_kv)
  int64_t max_partials;
  int32_t bt_stride, num_rows, num_tokens, num_pages;
  int32_t H_q, H_kv, D, G;
  int32_t dec_workers;       // decode worker warps in the grid
  int32_t num_sms;
  int32_t clear_status;      // the prologue zeroes the status word first (scratch owned by the library)
  int32_t force_chunk_ctas;  // test hook: CTAs that start on chunk work (-1: the cost model decides)
  float sm_mhz;              // cost model: the SM clock when no call has measured it yet,
  float hbm_gbs;             // and the HBM bandwidth that caps decode
  float l2_bytes;            // L2 capacity (orders the chunk items)
  float tile_cycles;         // cost model: SM cycles per 128x128 chunk tile,
  float dec_bytes_cycle;     // decode bytes per SM cycle,
  float key_bytes;           // and bytes of one key (K and V) of one KV head
  float scale_log2;
  int32_t* dec_rows;
  int32_t* dec_part_base;
  int32_t* dec_nsplit;
  int32_t* ch_rows;
  int2* dec_items;  // per decode split (items / H_kv entries): (decode row index, split within the row)
  int32_t* dec_cnt; // per (decode row, KV head): splits finished, for the last one to merge
  int2* ch_items;   // per chunk item: (chunk row index, KV head << 16 | Q-tile pair counted from the last)
  // the attention kernel's alone
  const bf16* q_rot;
  const uint8_t* kv_q4;   // 4-bit pool (q4.cuh), in the calls that take one
  const int32_t* bt;      // padded rows of bt_stride entries, or (bt_off given) every row's pages back to back
  bf16* out;
  float* part_ml;
  float* part_acc;
  uint64_t wait_limit_ns;  // bound of every chunk-phase wait
  int32_t test_stall;      // test hook: chunk-phase producers publish no work item, decode warps over a
                           // 4-bit pool issue no copy (0 in every real call)
  // chunk items in parts (4-bit pools), in what the workspace has behind its layout: room for ch_cap
  // parts of ch_rec query rows (ChunkParts)
  uint8_t* ch_parts;
  int32_t ch_cap, ch_rec;
};

// Where the parts' records lie: sums of O first ([part][row][D]), (max, sum)
// ([part][row]), the parts' table, then counters per item and Q tile.
struct ChunkParts {
  float* acc;
  float2* ml;
  int2* items;
  int32_t* cnt;
  __device__ __forceinline__ explicit ChunkParts(const AttnParams& p) {
    const int64_t rows = static_cast<int64_t>(p.ch_cap) * p.ch_rec;
    acc = reinterpret_cast<float*>(p.ch_parts);
    ml = reinterpret_cast<float2*>(p.ch_parts + rows * p.D * 4);
    items = reinterpret_cast<int2*>(p.ch_parts + rows * (p.D * 4 + 8));
    cnt = reinterpret_cast<int32_t*>(items + p.ch_cap);
  }
};

__host__ __device__ inline int64_t cdiv64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// first block-table entry of row `row`: padded rows or ragged offsets
__device__ __forceinline__ const int32_t* row_table(const AttnParams& p, int row) {
  return p.bt + (p.bt_off != nullptr ? static_cast<int64_t>(__ldg(p.bt_off + row))
                                     : static_cast<int64_t>(row) * p.bt_stride);
}

// ----------------------------------------------------------------------------
// prologue: validate, classify, order longest-first, lay out the work lists
// ----------------------------------------------------------------------------

// Exclusive scan of one int per thread over the block (blockDim.x a multiple
// of 32); returns the thread's prefix and sets `total`.  Each thread adds up
// the warp totals ahead of its own warp, so a scan costs two barriers.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_warp[w] = x;
  __syncthreads();
  int before = 0, tot = 0;
  for (int j = 0; j < nw; ++j) {
    const int t = s_warp[j];
    before += j < w ? t : 0;
    tot += t;
  }
  __syncthreads();  // s_warp is free again
  total = tot;
  return before + x - v;
}

// warp sum of values in [0, 2^31): two 32-bit reductions of the 16-bit halves
__device__ __forceinline__ int64_t warp_sum31(int v) {
  const unsigned lo = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v) & 0xffffu);
  const unsigned hi = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(v) >> 16);
  return (static_cast<int64_t>(hi) << 16) + lo;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Work items of one row: decode splits of `split` pages, or pairs of 128-row Q tiles.
__device__ __forceinline__ int row_items(bool chunk, int c, int d, int tpt, unsigned split) {
  if (!chunk) return static_cast<int>((static_cast<unsigned>(c + kPage) / kPage + split - 1) / split);
  const int n_qt = (d + tpt - 1) / tpt;
  return (n_qt + 1) >> 1;
}

constexpr int kChunkTile = 64;  // keys per KV tile of a chunk item
constexpr int kMinPartedTiles = 15;  // items of up to this many are not cut (chunk_part_tiles would not cut them)

// Parts of a chunk row's items, of `tiles` KV tiles or fewer each.
__device__ __forceinline__ int chunk_parts(int c, int d, int tiles) {
  return static_cast<int>((static_cast<unsigned>(c + d + kChunkTile - 1) / kChunkTile + tiles - 1) / tiles);
}

// 128x128 tiles of a chunk row's Q tiles against their causal key ranges (the
// cost model's unit of chunk work)
__device__ __forceinline__ unsigned chunk_tiles(int c, int d, int tpt) {
  unsigned tiles = 0;
  for (int end = tpt; end - tpt < d; end += tpt) tiles += static_cast<unsigned>(c + min(d, end) + 127) >> 7;
  return tiles;
}

// Sort key of the row at position `pos` of its list: the top 19 bits of the
// row's cost as a float (keys to read for a decode, query-key pairs for a
// chunk), then the position reversed.  Keys are unique and nonzero (cost >= 1);
// a larger key means more work or, at about equal cost, an earlier row.
__device__ __forceinline__ uint32_t order_key(float cost, int pos) {
  return ((__float_as_uint(cost) >> 13) << 13) | static_cast<uint32_t>(kMaxRows - 1 - pos);
}

// 32-bit words of the prologue's dynamic shared memory for S rows: sort keys
// (both lists, each padded to 4), list order, each row's d and c, and the item
// prefix in queue order.
__host__ __device__ constexpr int prologue_words(int S) { return 5 * ((S + 3) & ~3) + 16; }

// How many CTAs of the main kernel start on chunk tiles, and which side bounds
// the step.  Chunk time falls as 1/n with n chunk CTAs, in whole items; decode
// time is bytes over the bandwidth of the other SMs, capped by HBM.  Take the
// best split near the balance point, or, while decode stays HBM-bound, as many
// chunk CTAs as keep it so.  Called by one whole warp; the candidate counts go
// one per lane.
//
// It also orders the chunk items.  Longest first by default.  But when decode
// rows stream through L2 beside chunk rows whose K/V (all KV heads) would fill
// more than half of it, the items run KV head by KV head instead: the CTAs on
// chunk work at any time then share one head's K/V tiles in L2, where with
// every head in flight each head's prefix would be pulled from DRAM again and
// again (measured: 7 % more DRAM traffic than the algorithmic bytes on a
// 32K-key chunk next to 512 decodes, 6 % on 40 heads of 4K keys; on 8 heads
// of 10K keys, where the chunk rows bound the step, longest-first is faster).
struct SmSplit {
  int chunk_ctas;
  bool head_major;
};

__device__ SmSplit chunk_cta_split(const AttnParams& p, float tiles, float dec_pages, int n_items,
                                   int n_dec_items, float chunk_keys, int measured, int lane) {
  // the SM clock of the previous call on this workspace (header word H_CLOCK_MHZ, read
  // by the caller early), else the device's rated clock
  const float mhz = measured >= 200 && measured <= 5000 ? static_cast<float>(measured) : p.sm_mhz;
  const float S = static_cast<float>(p.num_sms);
  const float T = tiles * __fdividef(p.tile_cycles * 1000.f, mhz);  // SM-ns of chunk work
  const float B = dec_pages * p.H_kv * kPage * p.key_bytes;         // decode bytes
  const float g = p.dec_bytes_cycle * mhz * 1e-3f;                  // GB/s per decode SM
  const float n_hbm = fmaxf(0.f, floorf(S - p.hbm_gbs / g));  // most chunk CTAs with decode at HBM rate
  SmSplit r;
  r.head_major = B > 0.f && chunk_keys * p.H_kv * p.key_bytes > 0.5f * p.l2_bytes;
  // a step whose chunk items and decode items all start at once: a CTA per chunk item
  const int dec_ctas = static_cast<int>((static_cast<int64_t>(n_dec_items) * p.num_sms + p.dec_workers - 1) /
                                        p.dec_workers);
  if (n_items + dec_ctas <= p.num_sms) {
    r.chunk_ctas = n_items;
  } else if (T == 0.f) {
    r.chunk_ctas = static_cast<int>(B == 0.f ? S : n_hbm);
  } else if (B == 0.f) {
    r.chunk_ctas = static_cast<int>(S);
  } else if (T * p.hbm_gbs <= B * n_hbm) {  // chunk done within the HBM-bound decode time
    r.chunk_ctas = static_cast<int>(n_hbm);
  } else {
    // Balance point, then the nearby CTA count that minimizes the step: chunk work
    // comes in whole items, so n chunk CTAs need ceil(items / n) rounds of about
    // T / items each; decode runs on the other CTAs, capped by HBM.  Ties go to
    // the smallest count.
    const float n0 = fminf(S - 1.f, fmaxf(1.f, rintf(__fdividef(T * g * S, B + T * g))));
    const int n_it = max(n_items, 1);
    const float t_item = __fdividef(T, static_cast<float>(n_it));
    const int k_lo = max(1, static_cast<int>(n0) - 16), k_hi = min(static_cast<int>(S) - 1, static_cast<int>(n0) + 16);
    float best = 3.0e38f;
    int bk = static_cast<int>(n0);
    for (int k = k_lo + lane; k <= k_hi; k += 32) {
      const float tc = static_cast<float>((n_it + k - 1) / k) * t_item;
      const float td = __fdividef(B, fminf((S - k) * g, p.hbm_gbs));
      const float tt = fmaxf(tc, td);
      if (tt < best) {
        best = tt;
        bk = k;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int ok = __shfl_xor_sync(0xffffffffu, bk, o);
      if (ob < best || (ob == best && ok < bk)) {
        best = ob;
        bk = ok;
      }
    }
    r.chunk_ctas = bk;
  }
  if (p.force_chunk_ctas >= 0) r.chunk_ctas = min(p.force_chunk_ctas, p.num_sms);
  return r;
}

// Table entry of item i of a chunk row with np Q-tile pairs: (KV head) << 16 |
// (pair counted from the last), KV head by KV head or longest pair first.
__device__ __forceinline__ int chunk_entry(int i, int np, int H_kv, bool head_major) {
  const int hk = head_major ? i / np : i % H_kv;
  const int e = head_major ? i - hk * np : i / H_kv;
  return (hk << 16) | e;
}

// Decode split size: about 8 items per decode worker warp, clamped; at least 32
// pages (64 when G >= 4, whose items carry G heads of partials to merge, and 128
// when chunk rows share the step: decode then runs on the SMs the chunk tiles
// leave, where fewer, longer items cost less than a finer tail saves).
__device__ __forceinline__ int decode_split(const AttnParams& p, int64_t dec_pages, bool with_chunks) {
  const int64_t num = dec_pages * p.H_kv, den = static_cast<int64_t>(p.dec_workers) * 8;
  int64_t split = num + den <= 0xffffffffll
                      ? static_cast<int64_t>(static_cast<uint32_t>(num + den - 1) / static_cast<uint32_t>(den))
                      : cdiv64(num, den);
  const int64_t min_split = p.G >= 4 ? (with_chunks ? 4 : 2) * kMinSplitPages : kMinSplitPages;
  split = split < min_split ? min_split : (split > kMaxSplitPages ? kMaxSplitPages : split);
  return static_cast<int>(split);
}

// Split and team size of decode rows that teams of 2, 4, 8 or 16 warps of a CTA
// share split by split.  An estimate in microseconds for every pair of a team
// size (lane / 8) and a split (lane % 8), the smallest wins:
//     o max(1, x) + max(c P / W + 0.21 L, 0.45 L y) + 0.09 n max(1, G / team)
// x: splits over teams; y: x, rounded up while there are two rounds at most;
// P / W: pages per warp; L = min(split, longest row) / team: pages of a warp's
// share; n: splits of the longest row, which one team joins; o = 16, 11, 9, 9.4 by
// team size: the cost of a split around its pages; c = 1.15: a page's with the
// SM full at D = 128 (used at 64 too, where a page is half the work).  Fitted to
// sweeps of 27 pairs over 28 steps (1 to 512 rows of 1 to 32 KV heads, 1 to 131072
// keys, 19 to 420 us) in a build that forced the pair for the purpose: its choice was
// 2.3 % slower than the best pair on average, 11 % but for one step (4 rows of 64K to
// 128K keys: 20 %).  Called by whole warps.
struct DecPlan {
  int split, team;
};

// The pair that lane `lane` tries: 2, 4, 8, 16, 24, 32, 48 or 80 pages to a warp
// (and 128 in teams of 2 and 4) that give a team 32 pages or more, which the
// workspace's item and record counts allow.
__device__ __forceinline__ DecPlan dec_candidate(int lane) {
  const int small = 3 - (lane >> 3);  // sizes left out for this team
  uint64_t sizes = 0x5030201810080402ull;
  if (small > 0) sizes = (sizes >> (8 * small)) | ((small == 1 ? 0x5050505050505050ull : 0x8080808080808080ull) << (64 - 8 * small));
  const int per_warp = static_cast<int>(sizes >> (8 * (lane & 7))) & 255;
  const int team = 2 << (lane >> 3);
  return {team * per_warp, team};
}

template <bool Teams>
__device__ __forceinline__ DecPlan decode_plan(const AttnParams& p, int64_t dec_pages, int n_dec, int max_pages,
                                               bool with_chunks) {
  if (!Teams || n_dec == 0) return {decode_split(p, dec_pages, with_chunks), 1};
  const int lane = threadIdx.x & 31;
  const DecPlan cand = dec_candidate(lane);
  const float team = static_cast<float>(cand.team), split = static_cast<float>(cand.split);
  const float P = static_cast<float>(dec_pages) * p.H_kv, n = static_cast<float>(n_dec);
  const float W = static_cast<float>(p.dec_workers), mx = static_cast<float>(max_pages);
  const float splits = fmaxf(n, __fdividef(static_cast<float>(dec_pages), split) + 0.5f * n) * p.H_kv;
  const float x = __fdividef(splits * team, W), y = x <= 2.f ? ceilf(x) : x;
  const float L = __fdividef(fminf(split, mx), team);
  const float o = cand.team == 2 ? 16.f : cand.team == 4 ? 11.f : cand.team == 8 ? 9.f : 9.4f;
  const float t = o * fmaxf(1.f, x) + fmaxf(1.15f * __fdividef(P, W) + 0.21f * L, 0.45f * L * y) +
                  0.09f * __fdividef(mx, split) * fmaxf(1.f, __fdividef(static_cast<float>(p.G), team));
  const unsigned best = __reduce_min_sync(0xffffffffu, (__float_as_uint(t) & ~31u) | static_cast<unsigned>(lane));
  return dec_candidate(static_cast<int>(best & 31u));
}

// KV tiles to a part of a chunk item, or 0 for whole items.  Items are cut where
// they are fewer than half the CTAs that chunk work gets beside the decodes (k,
// the balance of chunk_cta_split): every part then starts at once.  Parts are
// written out and the last one to finish joins them, which costs about 0.0125 us a
// part and row where a tile takes about 1 us (D = 128), hence the square root; 8 tiles and a
// 32nd of the longest item at least, and only for a fifth of its time or more.
// pairs, pair_tiles: of one KV head, over the rows (a Q tile alone takes about the
// time of a pair).  32 / 8 heads, D = 128, whole (on a workspace without the room) and
// in parts: 20 tokens at 28000 347 and 71 us, 4 at 100000 1217 and 97 us, 128 at 8000
// beside 16 decodes of 512 to 8012 keys 131 and 81 us, four rows of 32 at 3000 to 6000
// 85 and 53 us.
__device__ __forceinline__ int chunk_part_tiles(const AttnParams& p, float pairs, float pair_tiles, float longest,
                                                float dec_pages) {
  const float n0 = pairs * p.H_kv, work = pair_tiles * p.H_kv;
  const float T = work * __fdividef(p.tile_cycles * 1000.f, p.sm_mhz), g = p.dec_bytes_cycle * p.sm_mhz * 1e-3f;
  const float B = dec_pages * p.H_kv * kPage * p.key_bytes;
  const float k = fminf(p.num_sms * __fdividef(T * g, B + T * g), static_cast<float>(p.ch_cap)) - 1.f;
  if (!(n0 >= 1.f && 2.f * n0 <= k)) return 0;
  const float row_us = 0.0125f * min(p.ch_rec, 128);
  const float tiles = ceilf(fmaxf(fmaxf(8.f, longest * (1.f / 32)), fmaxf(__fdividef(work, k - n0), sqrtf(row_us * longest))));
  const float cut = tiles + row_us * (__fdividef(longest, tiles) + 4.f) + 4.f;
  return cut < 0.8f * longest ? static_cast<int>(tiles) : 0;
}

// chunk_part_tiles for a chunk row per lane (keys: its context, or 0; np: its pairs).
__device__ __noinline__ int plan_parts_warp(const AttnParams& p, int keys, int np, int64_t dec_pages) {
  const int n_kt = (keys + kChunkTile - 1) / kChunkTile, longest = __reduce_max_sync(0xffffffffu, n_kt);
  if (longest <= kMinPartedTiles) return 0;
  const int64_t pair_tiles = warp_sum31(static_cast<int>(min(static_cast<int64_t>(np) * n_kt, int64_t{0x7fffffff})));
  return chunk_part_tiles(p, static_cast<float>(__reduce_add_sync(0xffffffffu, np)), static_cast<float>(pair_tiles),
                          static_cast<float>(longest), static_cast<float>(dec_pages));
}

// chunk_part_tiles for the rows of a block, from their values in shared memory.  Called by every
// thread.  Both forms are out of line: the prologue runs from a cold instruction cache, and most
// steps need neither.
__device__ __noinline__ int plan_parts_block(const AttnParams& p, const int* rd, const int* rc, int64_t dec_pages) {
  __shared__ long long s_tiles[32];
  __shared__ int s_pairs[32], s_longest[32];
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  int64_t tiles = 0;
  int pairs = 0, longest = 0;
  for (int s = tid; s < p.num_rows; s += nt) {
    const int c = rc[s], d = rd[s];
    if (d <= 1) continue;
    const int np = row_items(true, c, d, 128 / p.G, 1u), n_kt = chunk_parts(c, d, 1);
    pairs += np;
    tiles += static_cast<int64_t>(np) * n_kt;
    longest = max(longest, n_kt);
  }
  tiles = warp_sum64(tiles);
  pairs = __reduce_add_sync(0xffffffffu, pairs);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) {
    s_tiles[warp] = tiles;
    s_pairs[warp] = pairs;
    s_longest[warp] = longest;
  }
  __syncthreads();
  tiles = pairs = longest = 0;
  for (int j = 0; j < nw; ++j) {
    tiles += s_tiles[j];
    pairs += s_pairs[j];
    longest = max(longest, s_longest[j]);
  }
  if (longest <= kMinPartedTiles) return 0;
  return chunk_part_tiles(p, static_cast<float>(pairs), static_cast<float>(tiles), static_cast<float>(longest),
                          static_cast<float>(dec_pages));
}

// Table entries and counters of a chunk row in parts, from place `first`: `items` of
// them per KV head, the parts of a pair neighbours.  The first word is the row's
// position k in the list and, above it, the part.  By one warp.
__device__ __noinline__ void chunk_part_table(const AttnParams& p, int first, int k, int items, int parts, bool head_major,
                                              int lane) {
  const ChunkParts cp(p);
  for (int i = lane; i < items * p.H_kv; i += 32) {
    const int j = i / parts;
    cp.items[first + i] = make_int2(k | ((i - j * parts) << 16), chunk_entry(j, items / parts, p.H_kv, head_major));
    reinterpret_cast<int2*>(cp.cnt)[first + i] = make_int2(0, 0);
  }
}

// First word of a decode row's table entries: its position k in the list, and for
// teams, which look every word of a split up at once, its row above that.
template <bool Teams>
__device__ __forceinline__ int dec_entry(int k, int row) {
  return Teams ? k | (row << 16) : k;
}

// Warps that the decode items keep busy at a time, at most.
__device__ __forceinline__ int dec_item_warps(int64_t items, int team) {
  const int64_t n = items * team;
  return n < 0x7fffffff ? static_cast<int>(n) : 0x7fffffff;
}

// Header of a call whose metadata failed validation: status set, no work.
__device__ __forceinline__ void header_bad_meta(int32_t* hdr) {
  atomicOr(hdr + H_STATUS, MS_STATUS_BAD_META);
  hdr[H_DEC_CTR] = hdr[H_CH_CTR] = 0;
  hdr[H_NDEC] = hdr[H_NDEC_ITEMS] = hdr[H_NCH] = hdr[H_NCH_ITEMS] = hdr[H_NPART] = 0;
  hdr[H_SPLIT] = kMinSplitPages;
  hdr[H_CHUNK_CTAS] = 0;
}

// The prologue of a step of at most 32 rows: one warp, a row per lane, with
// ballots and shuffles in place of shared memory and barriers.  Same outputs
// as the block version below.
template <bool Teams>
__device__ __forceinline__ void prologue_warp(const AttnParams& p) {
  const int lane = threadIdx.x, S = p.num_rows;
  int32_t* hdr = p.hdr;
  const int measured_mhz = hdr[H_CLOCK_MHZ];  // loaded beside the row metadata
  int d = 0, c = 0, ctx = 0;
  bool ok = true;
  if (lane < S) {
    const int32_t a = p.cu[lane], b = p.cu[lane + 1];
    d = static_cast<int32_t>(static_cast<uint32_t>(b) - static_cast<uint32_t>(a));  // checked below
    c = p.q_start[lane];
    ctx = p.ctx_lens[lane];
    ok = a >= 0 && b >= a && b <= p.num_tokens && c >= 0 && static_cast<int64_t>(ctx) == static_cast<int64_t>(c) + d;
    if (p.bt_off != nullptr) {
      const int64_t o0 = p.bt_off[lane], o1 = p.bt_off[lane + 1];
      ok = ok && o0 >= 0 && o1 <= p.bt_len && cdiv64(ctx, kPage) <= o1 - o0;
    } else {
      ok = ok && cdiv64(ctx, kPage) <= p.bt_stride;
    }
    if (!ok) d = ctx = 0;
  }
  const bool bad = __any_sync(0xffffffffu, !ok);
  const int64_t ctx_sum = warp_sum31(ctx);  // ctx >= 0 here (valid rows, or 0)
  if (bad || ctx_sum > p.context_total) {
    if (lane == 0) header_bad_meta(hdr);
    return;
  }
  const bool is_dec = d == 1, is_ch = d > 1;
  const int64_t dec_pages = warp_sum31(is_dec ? (ctx + kPage - 1) / kPage : 0);
  const int tpt = 128 / p.G;
  const unsigned bd = __ballot_sync(0xffffffffu, is_dec), bc = __ballot_sync(0xffffffffu, is_ch);
  const int n_dec = __popc(bd), n_ch = __popc(bc);
  const int max_pages = Teams ? __reduce_max_sync(0xffffffffu, is_dec ? (ctx + kPage - 1) / kPage : 0) : 0;
  const DecPlan plan = decode_plan<Teams>(p, dec_pages, n_dec, max_pages, n_ch > 0);
  const int split = plan.split;
  // position in its list, then rank by key within the list (longest first):
  // the keys sit in shared memory by list position, zero-padded, read 16 bytes at a time
  __shared__ __align__(16) uint32_t s_key[2][32];
  __shared__ int s_items[32], s_pref[32];
  const bool listed = is_dec || is_ch;
  const unsigned list = is_ch ? bc : bd;
  const int pos = __popc(list & ((1u << lane) - 1u));
  const uint32_t key = order_key(is_ch ? 0.5f * d * (2.f * c + d + 1.f) : c + 1.f, pos);
  s_key[0][lane] = 0;
  s_key[1][lane] = 0;
  s_items[lane] = 0;
  __syncwarp();
  if (listed) s_key[is_ch][pos] = key;
  __syncwarp();
  int rank = 0;
  const uint4* k4 = reinterpret_cast<const uint4*>(s_key[is_ch]);
#pragma unroll
  for (int m = 0; m < 8; ++m) {
    const uint4 v = k4[m];
    rank += (v.x > key) + (v.y > key) + (v.z > key) + (v.w > key);
  }
  int part_tiles = 0, parts = 1;
  int items = listed ? row_items(is_ch, c, d, tpt, static_cast<unsigned>(split)) : 0;
  if (Teams && 2 * n_ch * p.H_kv < p.num_sms &&  // the least that chunk_part_tiles needs
      __reduce_max_sync(0xffffffffu, is_ch ? ctx : 0) > kMinPartedTiles * kChunkTile) {
    part_tiles = plan_parts_warp(p, is_ch ? ctx : 0, is_ch ? items : 0, dec_pages);
    if (part_tiles > 0 && is_ch) items *= parts = chunk_parts(c, d, part_tiles);
  }
  const int q = (is_ch ? n_dec : 0) + rank;  // queue position
  if (listed) s_items[q] = items;
  __syncwarp();
  {  // exclusive prefix over queue positions, one per lane
    const int v = s_items[lane];
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    s_pref[lane] = x - v;
  }
  __syncwarp();
  const int before = listed ? s_pref[q] : 0;  // items of the rows ahead in queue order
  const int dec_tot = __reduce_add_sync(0xffffffffu, is_dec ? items : 0);
  const int ch_tot = __reduce_add_sync(0xffffffffu, is_ch ? items : 0);
  const int64_t n_dec_items = static_cast<int64_t>(dec_tot) * p.H_kv;
  const int64_t n_ch_items = static_cast<int64_t>(ch_tot) * p.H_kv;
  const bool dec_over = n_dec_items > p.max_dec_items || static_cast<int64_t>(dec_tot) * p.H_q > p.max_partials;
  const bool ch_over = n_ch_items > (part_tiles > 0 ? p.ch_cap : p.max_ch_items);
  const int64_t tiles =
      warp_sum31(is_ch ? static_cast<int>(min(static_cast<int64_t>(chunk_tiles(c, d, tpt)) * p.H_kv,
                                                int64_t{0x7fffffff}))
                       : 0);
  const int64_t chunk_keys = warp_sum31(is_ch ? ctx : 0);
  if (is_dec) {
    p.dec_rows[rank] = lane;
    p.dec_part_base[rank] = static_cast<int32_t>(static_cast<int64_t>(before) * p.H_q);
    p.dec_nsplit[rank] = items;
    if (!dec_over)
      for (int i = 0; i < items; ++i) p.dec_items[before + i] = make_int2(dec_entry<Teams>(rank, lane), i);
  }
  if (is_ch) p.ch_rows[rank] = lane;
  const SmSplit sp = chunk_cta_split(p, static_cast<float>(tiles), static_cast<float>(dec_pages),
                                     ch_over ? 0 : static_cast<int>(n_ch_items),
                                     dec_over ? 0 : dec_item_warps(n_dec_items, plan.team), static_cast<float>(chunk_keys),
                                     measured_mhz, lane);
  // the chunk rows' items (pairs x H_kv of them per row), the whole warp on one row at
  // a time; then the split counters, 16 bytes per store
  for (unsigned pend = ch_over ? 0u : bc; pend != 0u; pend &= pend - 1u) {
    const int src = __ffs(pend) - 1;
    const int r_rank = __shfl_sync(0xffffffffu, rank, src), r_items = __shfl_sync(0xffffffffu, items, src);
    const int r_before = __shfl_sync(0xffffffffu, before, src);
    if (Teams && part_tiles > 0) {
      chunk_part_table(p, (r_before - dec_tot) * p.H_kv, r_rank, r_items, __shfl_sync(0xffffffffu, parts, src), sp.head_major,
                       lane);
      continue;
    }
    int2* out = p.ch_items + static_cast<int64_t>(r_before - dec_tot) * p.H_kv;
    for (int i = lane; i < r_items * p.H_kv; i += 32)
      out[i] = make_int2(r_rank, chunk_entry(i, r_items, p.H_kv, sp.head_major));
  }
  if (!dec_over) {
    const int n_cnt = n_dec * p.H_kv;  // the counters start 16-byte aligned in the workspace
    for (int i = lane; i < (n_cnt >> 2); i += 32) reinterpret_cast<int4*>(p.dec_cnt)[i] = make_int4(0, 0, 0, 0);
    for (int i = (n_cnt & ~3) + lane; i < n_cnt; i += 32) p.dec_cnt[i] = 0;
  }
  if (lane == 0) {
    hdr[H_NDEC] = dec_over ? 0 : n_dec;
    hdr[H_NDEC_ITEMS] = dec_over ? 0 : static_cast<int32_t>(n_dec_items);
    hdr[H_NPART] = static_cast<int32_t>(static_cast<int64_t>(dec_tot) * p.H_q);
    hdr[H_NCH] = ch_over ? 0 : n_ch;
    hdr[H_NCH_ITEMS] = ch_over ? 0 : static_cast<int32_t>(n_ch_items);
    if (dec_over || ch_over) atomicOr(hdr + H_STATUS, MS_STATUS_BAD_META);
    hdr[H_DEC_CTR] = 0;
    hdr[H_CH_CTR] = 0;
    hdr[H_SPLIT] = split;
    if (Teams) {
      hdr[H_TEAM] = plan.team;
      hdr[H_CH_TILES] = part_tiles;
    }
    hdr[H_CHUNK_CTAS] = sp.chunk_ctas;
  }
}

// The prologue on one CTA of blockDim.x threads (a multiple of 32, at most
// 1024; warp 0 alone up to 32 rows): validate the rows, split them into decode rows (d = 1)
// and chunk rows (d > 1), order each list longest-first, size the decode
// splits, write the flat item tables (item -> row in queue order, item within
// the row), zero the split counters and pick how many CTAs of the main kernel
// start on chunk work.  Every row's values are read from global memory once;
// the rest happens in shared memory (prologue_words(S) words of dynamic shared
// memory).  It runs once per step from a cold instruction cache, so its loops
// stay rolled and its code short.  It reads only the row metadata, never the
// appended K/V, so it may run alongside the append.
template <bool Teams>
__device__ __forceinline__ void prologue_body(const AttnParams& p) {
  extern __shared__ __align__(16) int32_t psm[];
  __shared__ int s_warp[32];
  __shared__ long long s_sum[3][32];
  __shared__ unsigned s_cnt[3][32];
  __shared__ unsigned long long s_tiles;
  __shared__ SmSplit s_split;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int S = p.num_rows;  // at most kMaxRows (checked by the host, which sizes psm by it)
  int32_t* hdr = p.hdr;
  const int Sp = (S + 3) & ~3;
  uint32_t* key = reinterpret_cast<uint32_t*>(psm);  // Sp + 8 words
  int32_t* lst = psm + Sp + 8;                       // list order: decode rows, then chunk rows
  int32_t* rd = lst + Sp;                            // per row (input order): d (0 for pad rows), c
  int32_t* rc = rd + Sp;
  int32_t* pref = rc + Sp;                           // per queue position: items, then their prefix
  // a library-owned scratch keeps the previous call's status: start this call at zero
  // (ahead of every status write of this call, all of which come after a barrier or from this thread)
  if (tid == 0 && p.clear_status) hdr[H_STATUS] = 0;
  if (S <= 32) {
    if (warp == 0) prologue_warp<Teams>(p);
    return;
  }
  if (tid == 0) s_tiles = 0;
  const int measured_mhz = warp == 0 ? hdr[H_CLOCK_MHZ] : 0;  // for the SM split, loaded early
  // 1. load and validate the rows; count decodes, chunks, context and decode pages
  int64_t my_ctx = 0, my_pages = 0, my_ch_keys = 0;
  unsigned my_dec = 0, my_ch = 0, my_max = 0;
  int my_bad = 0;
  for (int s = tid; s < S; s += nt) {
    const int32_t a = p.cu[s], b = p.cu[s + 1];
    const int32_t d = static_cast<int32_t>(static_cast<uint32_t>(b) - static_cast<uint32_t>(a));  // checked below
    const int32_t c = p.q_start[s], ctx = p.ctx_lens[s];
    // d == 0 is a pad row: valid, and neither a decode nor a chunk
    bool ok = a >= 0 && b >= a && b <= p.num_tokens && c >= 0 && static_cast<int64_t>(ctx) == static_cast<int64_t>(c) + d;
    if (p.bt_off != nullptr) {  // the row's pages must lie inside the table
      const int64_t o0 = p.bt_off[s], o1 = p.bt_off[s + 1];
      ok = ok && o0 >= 0 && o1 <= p.bt_len && cdiv64(ctx, kPage) <= o1 - o0;
    } else {
      ok = ok && cdiv64(ctx, kPage) <= p.bt_stride;
    }
    my_bad |= !ok;
    rd[s] = ok ? d : 0;
    rc[s] = c;
    if (ok) {
      my_ctx += ctx;
      my_dec += d == 1;
      my_ch += d > 1;
      if (d == 1) {
        const unsigned n = static_cast<unsigned>(ctx + kPage - 1) / kPage;
        my_pages += n;
        my_max = max(my_max, n);
      }
      if (d > 1) my_ch_keys += ctx;
    }
  }
  my_ctx = warp_sum64(my_ctx);
  my_pages = warp_sum64(my_pages);
  my_ch_keys = warp_sum64(my_ch_keys);
  my_dec = __reduce_add_sync(0xffffffffu, my_dec);
  my_ch = __reduce_add_sync(0xffffffffu, my_ch);
  if (Teams) my_max = __reduce_max_sync(0xffffffffu, my_max);
  if (lane == 0) {
    s_sum[0][warp] = my_ctx;
    s_sum[1][warp] = my_pages;
    s_sum[2][warp] = my_ch_keys;
    s_cnt[0][warp] = my_dec;
    s_cnt[1][warp] = my_ch;
    if (Teams) s_cnt[2][warp] = my_max;
  }
  const int bad = __syncthreads_or(my_bad);
  int64_t ctx_sum = 0, dec_pages = 0, chunk_keys = 0;
  int n_dec = 0, n_ch = 0, max_pages = 0;
  for (int j = 0; j < nw; ++j) {
    ctx_sum += s_sum[0][j];
    dec_pages += s_sum[1][j];
    chunk_keys += s_sum[2][j];
    n_dec += static_cast<int>(s_cnt[0][j]);
    n_ch += static_cast<int>(s_cnt[1][j]);
    if (Teams) max_pages = max(max_pages, static_cast<int>(s_cnt[2][j]));
  }
  if (bad || ctx_sum > p.context_total) {
    if (tid == 0) header_bad_meta(hdr);
    return;
  }
  // 2. decode split size
  const DecPlan plan = decode_plan<Teams>(p, dec_pages, n_dec, max_pages, n_ch > 0);
  const int split = plan.split;
  const int part_tiles = Teams && 2 * n_ch * p.H_kv < p.num_sms && chunk_keys > kMinPartedTiles * kChunkTile &&
                                 (p.cu[S] - n_dec) / 128 * p.G * p.H_kv < p.num_sms  // the least that it needs
                             ? plan_parts_block(p, rd, rc, dec_pages) : 0;
  const int tpt = 128 / p.G;
  const unsigned split32 = static_cast<unsigned>(split);
  // 3. the two lists in input order: decode rows at lst[0, n_dec), chunk rows after them
  const int n_tot = n_dec + n_ch;
  {
    int o_dec = 0, o_ch = 0;
    for (int base = 0; base < S; base += nt) {  // uniform
      const int s = base + tid;  // the row this thread loaded
      const int d = s < S ? rd[s] : 0;
      int tot;
      const int o = block_scan((d == 1) | ((d > 1) << 16), s_warp, tot);  // both counts, 16 bits each
      if (d == 1) lst[o_dec + (o & 0xffff)] = s;
      if (d > 1) lst[n_dec + o_ch + (o >> 16)] = s;
      o_dec += tot & 0xffff;
      o_ch += tot >> 16;
    }
  }
  // 4. sort keys, each list from a 16-byte boundary, padded with zero keys
  const int ch_base = (n_dec + 3) & ~3;
  if (tid < 4) {
    if (n_dec + tid < ch_base) key[n_dec + tid] = 0;
    if (n_ch + tid < ((n_ch + 3) & ~3)) key[ch_base + n_ch + tid] = 0;
  }
  __syncthreads();
  for (int j = tid; j < n_tot; j += nt) {
    const bool ch = j >= n_dec;
    const int pos = ch ? j - n_dec : j, row = lst[j];
    const float d = static_cast<float>(rd[row]), c = static_cast<float>(rc[row]);
    key[(ch ? ch_base : 0) + pos] = order_key(ch ? 0.5f * d * (2.f * c + d + 1.f) : c + 1.f, pos);
  }
  __syncthreads();
  // 5. each list longest first: a row's rank is the number of larger keys in its
  // list (lists longer than kSortLimit keep input order); rows in queue order,
  // and each row's item count at its queue position
  for (int j = tid; j < n_tot; j += nt) {
    const bool ch = j >= n_dec;
    const int pos = ch ? j - n_dec : j, n = ch ? n_ch : n_dec;
    int rank = pos;
    if (n <= kSortLimit) {
      const uint32_t* kl = key + (ch ? ch_base : 0);
      const uint32_t mine = kl[pos];
      const uint4* k4 = reinterpret_cast<const uint4*>(kl);
      rank = 0;
      for (int m = 0; m < (n + 3) >> 2; ++m) {
        const uint4 v = k4[m];
        rank += (v.x > mine) + (v.y > mine) + (v.z > mine) + (v.w > mine);
      }
    }
    const int row = lst[j], c = rc[row], d = rd[row];
    (ch ? p.ch_rows : p.dec_rows)[rank] = row;
    pref[(ch ? n_dec : 0) + rank] = row_items(ch, c, d, tpt, split32) * (Teams && ch && part_tiles > 0 ? chunk_parts(c, d, part_tiles) : 1);
    if (ch) atomicAdd(&s_tiles, static_cast<unsigned long long>(chunk_tiles(c, d, tpt)) * p.H_kv);
  }
  __syncthreads();
  // 6. exclusive prefix of the item counts in queue order (decode rows, then chunk rows)
  int run = 0;
  for (int base = 0; base < n_tot; base += nt) {  // uniform
    const int q = base + tid;
    const int v = q < n_tot ? pref[q] : 0;
    int tot;
    const int o = block_scan(v, s_warp, tot);
    if (q < n_tot) {
      pref[q] = run + o;
      if (q < n_dec) {
        p.dec_part_base[q] = static_cast<int32_t>(static_cast<int64_t>(run + o) * p.H_q);
        p.dec_nsplit[q] = v;
      }
    }
    run += tot;
  }
  if (tid == 0) pref[n_tot] = run;
  __syncthreads();
  const int dec_tot = pref[n_dec], ch_tot = run - dec_tot;
  const int64_t n_dec_items = static_cast<int64_t>(dec_tot) * p.H_kv;
  const int64_t n_ch_items = static_cast<int64_t>(ch_tot) * p.H_kv;
  const bool dec_over = n_dec_items > p.max_dec_items || static_cast<int64_t>(dec_tot) * p.H_q > p.max_partials;
  const bool ch_over = n_ch_items > (part_tiles > 0 ? p.ch_cap : p.max_ch_items);
  // 7. item tables.  Decode rows, a thread per row: entry pref[q] + i -> (row
  // k, split i), one entry per split (a work item is an entry and a KV head).
  // Then the SM split, which also orders the chunk items; chunk rows, a warp
  // per row: one entry per item, (row k, KV head and Q-tile pair).  Then the
  // split counters of every (decode row, KV head), zeroed 16 bytes at a time.
  for (int q = tid; q < n_dec && !dec_over; q += nt) {
    const int cnt = pref[q + 1] - pref[q];
    int2* out = p.dec_items + pref[q];
    const int x = dec_entry<Teams>(q, Teams ? p.dec_rows[q] : 0);
    for (int i = 0; i < cnt; ++i) out[i] = make_int2(x, i);
  }
  if (warp == 0) {
    const SmSplit sp = chunk_cta_split(p, static_cast<float>(s_tiles), static_cast<float>(dec_pages),
                                       ch_over ? 0 : static_cast<int>(n_ch_items),
                                       dec_over ? 0 : dec_item_warps(n_dec_items, plan.team), static_cast<float>(chunk_keys),
                                       measured_mhz, lane);
    if (lane == 0) s_split = sp;
  }
  __syncthreads();
  for (int q = n_dec + warp; q < n_tot && !ch_over; q += nw) {
    const int np = pref[q + 1] - pref[q];
    if (Teams && part_tiles > 0) {
      const int row = p.ch_rows[q - n_dec];
      chunk_part_table(p, (pref[q] - dec_tot) * p.H_kv, q - n_dec, np, chunk_parts(rc[row], rd[row], part_tiles),
                       s_split.head_major, lane);
      continue;
    }
    int2* out = p.ch_items + static_cast<int64_t>(pref[q] - dec_tot) * p.H_kv;
    for (int i = lane; i < np * p.H_kv; i += 32)
      out[i] = make_int2(q - n_dec, chunk_entry(i, np, p.H_kv, s_split.head_major));
  }
  if (!dec_over) {
    const int n_cnt = n_dec * p.H_kv;  // the counters start 16-byte aligned in the workspace
    for (int i = tid; i < (n_cnt >> 2); i += nt) reinterpret_cast<int4*>(p.dec_cnt)[i] = make_int4(0, 0, 0, 0);
    for (int i = (n_cnt & ~3) + tid; i < n_cnt; i += nt) p.dec_cnt[i] = 0;
  }
  // 8. the header the main kernel starts from
  if (warp == 0) {
    if (lane == 0) {
      hdr[H_NDEC] = dec_over ? 0 : n_dec;
      hdr[H_NDEC_ITEMS] = dec_over ? 0 : static_cast<int32_t>(n_dec_items);
      hdr[H_NPART] = static_cast<int32_t>(static_cast<int64_t>(dec_tot) * p.H_q);
      hdr[H_NCH] = ch_over ? 0 : n_ch;
      hdr[H_NCH_ITEMS] = ch_over ? 0 : static_cast<int32_t>(n_ch_items);
      if (dec_over || ch_over) atomicOr(hdr + H_STATUS, MS_STATUS_BAD_META);
      hdr[H_DEC_CTR] = 0;
      hdr[H_CH_CTR] = 0;
      hdr[H_SPLIT] = static_cast<int32_t>(split);
      if (Teams) {
        hdr[H_TEAM] = plan.team;
        hdr[H_CH_TILES] = part_tiles;
      }
      hdr[H_CHUNK_CTAS] = s_split.chunk_ctas;
    }
  }
}

// The prologue as its own kernel, launched as a programmatic dependent of the
// kernel before it on the stream (normally the append): it runs alongside that
// kernel and waits for it before it exits, so the kernel after it sees the
// append's writes.
template <bool Teams>
__global__ void __launch_bounds__(1024, 1) prologue_kernel(AttnParams p) {
  griddep_launch_dependents();
  prologue_body<Teams>(p);
  griddep_wait();
}

// Merge the ns split records of decode row k for query heads h0 .. h0+nh-1
// into bf16 output (one warp; lane owns D/32 columns).  Records written by
// other SMs are read past L1.  U: records in flight at a time.
template <int D, int U = 4>
__device__ __forceinline__ void merge_splits(const AttnParams& p, int k, int h0, int nh, int tok, int ns,
                                             int lane) {
  constexpr int EPL = D / 32;
  const int64_t base0 = __ldcg(p.dec_part_base + k);
  for (int hq = h0; hq < h0 + nh; ++hq) {
    const int64_t base = base0 + hq;
    // lanes over splits for (max, sum); then every lane walks the splits for its columns
    float M = -INFINITY;
    for (int j = lane; j < ns; j += 32)
      M = fmaxf(M, __ldcg(p.part_ml + (base + static_cast<int64_t>(j) * p.H_q) * 2));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float L = 0.f, o[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] = 0.f;
    for (int j0 = 0; j0 < ns; j0 += 32) {
      const int j = j0 + lane;
      float w = 0.f;
      if (j < ns) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + (base + static_cast<int64_t>(j) * p.H_q) * 2));
        w = ex2(ml.x - M);
        L += w * ml.y;
      }
      const int nj = min(32, ns - j0);
#pragma unroll U
      for (int jj = 0; jj < nj; ++jj) {
        const float wj = __shfl_sync(0xffffffffu, w, jj);
        const float* src = p.part_acc + (base + static_cast<int64_t>(j0 + jj) * p.H_q) * D + lane * EPL;
        if constexpr (EPL == 4) {
          const float4 a = __ldcg(reinterpret_cast<const float4*>(src));
          o[0] += wj * a.x; o[1] += wj * a.y; o[2] += wj * a.z; o[3] += wj * a.w;
        } else {
          const float2 a = __ldcg(reinterpret_cast<const float2*>(src));
          o[0] += wj * a.x; o[1] += wj * a.y;
        }
      }
    }
#pragma unroll
    for (int o2 = 16; o2 > 0; o2 >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o2);
    const float inv = 1.f / L;
    bf16* dst = p.out + (static_cast<int64_t>(tok) * p.H_q + hq) * D + lane * EPL;
    if constexpr (EPL == 4) {
      __nv_bfloat162 a = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
      __nv_bfloat162 b = __floats2bfloat162_rn(o[2] * inv, o[3] * inv);
      *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
    } else {
      __nv_bfloat162 a = __floats2bfloat162_rn(o[0] * inv, o[1] * inv);
      *reinterpret_cast<__nv_bfloat162*>(dst) = a;
    }
  }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------

struct WsLayout {
  size_t hdr, dec_rows, dec_part_base, dec_nsplit, ch_rows, dec_cnt, dec_items,
      ch_items, part_ml, part_acc, total;
  int64_t max_partials, max_dec_items, max_ch_items;
};

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline WsLayout ws_layout(int64_t max_rows, int64_t max_tokens, int64_t max_context_total, int64_t H_q, int64_t H_kv,
                   int64_t D) {
  WsLayout w;
  size_t off = 0;
  w.hdr = off;
  off += H_WORDS * 4;
  w.dec_rows = off;
  off = align_up(off + max_rows * 4, 16);
  w.dec_part_base = off;
  off = align_up(off + max_rows * 4, 16);
  w.dec_nsplit = off;
  off = align_up(off + max_rows * 4, 16);
  w.ch_rows = off;
  off = align_up(off + max_rows * 4, 16);
  w.dec_cnt = off;
  off = align_up(off + max_rows * H_kv * 4, 256);
  // every decode split covers >= kMinSplitPages pages: splits <= ctx / (16 * kMinSplitPages) + rows
  const int64_t max_splits = cdiv64(max_context_total, kPage * kMinSplitPages) + 2 * max_rows;
  const int64_t G = H_q / (H_kv > 0 ? H_kv : 1);
  w.max_dec_items = H_kv * max_splits;
  w.max_ch_items = H_kv * (cdiv64(max_tokens * G, 128) + max_rows);
  w.dec_items = off;  // one entry per split: the KV head is not in the table
  off = align_up(off + (w.max_dec_items / H_kv) * 8, 256);
  w.ch_items = off;  // one entry per chunk item
  off = align_up(off + w.max_ch_items * 8, 256);
  w.max_partials = H_q * max_splits;
  w.part_ml = off;
  off = align_up(off + w.max_partials * 2 * 4, 256);
  w.part_acc = off;
  off = align_up(off + w.max_partials * D * 4, 256);
  w.total = off;
  return w;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// the driver's tensor-map encoder, looked up once (thread-safe static initialisation)
inline EncodeTiledFn get_encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(ptr);
    return nullptr;
  }();
  return fn;
}

inline bool encode_bf16(EncodeTiledFn fn, CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                 const cuuint64_t* strides_bytes, const cuuint32_t* box) {
  cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides_bytes, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What a workspace holds behind its layout for chunk items in parts: bytes of one
// part of `rec` query rows (table entry, two counters, then (max, sum) and D sums a row),
// and of kPartItems of them, about one for every SM (of steps of at most max_tokens tokens).
constexpr int kPartItems = 152;

inline int part_rows(int64_t tokens, int64_t G) { return static_cast<int>(tokens * G < 256 ? tokens * G : 256); }

inline size_t part_bytes(int rec, int64_t D) { return 16 + static_cast<size_t>(rec) * (8 + 4 * static_cast<size_t>(D)); }

inline size_t parts_total(int64_t max_tokens, int64_t H_q, int64_t H_kv, int64_t D) {
  if (max_tokens < 2) return 0;
  return align_up(kPartItems * part_bytes(part_rows(max_tokens, H_q / H_kv), D), 256);
}

std::atomic<int> g_num_sms[kMaxDevices];

inline int num_sms() {
  const int dev = current_device();
  if (dev < 0) return -1;
  const int cached = g_num_sms[dev].load(std::memory_order_relaxed);
  if (cached > 0) return cached;
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return -1;
  g_num_sms[dev].store(n, std::memory_order_relaxed);
  return n;
}

// The cost model's device rates, looked up once per device: the rated SM
// clock (MHz) and the HBM bandwidth (GB/s), nominal (memory clock x bus width,
// double data rate) times the sustained copy share.
std::atomic<float> g_sm_mhz[kMaxDevices], g_hbm_gbs[kMaxDevices], g_l2_bytes[kMaxDevices];

inline int device_rates(float* sm_mhz, float* hbm_gbs, float* l2_bytes) {
  const int dev = current_device();
  if (dev < 0) return MS_ERR_CUDA;
  float mhz = g_sm_mhz[dev].load(std::memory_order_relaxed);
  float gbs = g_hbm_gbs[dev].load(std::memory_order_relaxed);
  float l2 = g_l2_bytes[dev].load(std::memory_order_relaxed);
  if (!(mhz > 0.f) || !(gbs > 0.f) || !(l2 > 0.f)) {
    int clk_khz = 0, mem_khz = 0, bus_bits = 0, l2_b = 0;
    if (cudaDeviceGetAttribute(&clk_khz, cudaDevAttrClockRate, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&mem_khz, cudaDevAttrMemoryClockRate, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&bus_bits, cudaDevAttrGlobalMemoryBusWidth, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&l2_b, cudaDevAttrL2CacheSize, dev) != cudaSuccess)
      return MS_ERR_CUDA;
    mhz = clk_khz > 0 ? clk_khz * 1e-3f : 2000.f;
    gbs = mem_khz > 0 && bus_bits > 0 ? 2.f * mem_khz * 1e3f * (bus_bits / 8.f) * 1e-9f * kHbmCopyEfficiency : 6500.f;
    l2 = l2_b > 0 ? static_cast<float>(l2_b) : 64.f * (1 << 20);
    g_sm_mhz[dev].store(mhz, std::memory_order_relaxed);
    g_hbm_gbs[dev].store(gbs, std::memory_order_relaxed);
    g_l2_bytes[dev].store(l2, std::memory_order_relaxed);
  }
  *sm_mhz = mhz;
  *hbm_gbs = gbs;
  *l2_bytes = l2;
  return MS_OK;
}

// Launch as a programmatic dependent of the previous kernel on the stream: the
// kernel may start while that one finishes and orders itself with
// griddepcontrol.wait.
template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                             Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks every argument of an attention call and fills *p; enqueues nothing.
// *empty: the step has no tokens, so there is nothing to launch.  The pools
// come as two pointers (one pool twice where K and V share it); what depends
// on their form -- tensor maps, decode workers, the cost model's rates -- is
// the caller's to fill in.  clear_status makes the prologue zero the status
// word before anything of this call can set it.  stall_limit_ns > 0 is the
// test hook of ms_test_attention_stall: chunk-phase producers publish nothing
// and every chunk-phase wait gives up after that many nanoseconds.
inline int step_setup(const void* q_rot, const void* k_cache, const void* v_cache, int32_t num_pages,
                      const int32_t* cu_seqlens_q, const int32_t* q_start_pos, const int32_t* context_lens,
                      const int32_t* block_tables, const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride,
                      int32_t num_rows, int32_t num_tokens, int64_t context_total, int32_t H_q, int32_t H_kv,
                      int32_t D, int32_t page_size, float scale, void* out, void* workspace, size_t ws_bytes,
                      bool clear_status, int64_t stall_limit_ns, AttnParams* params, bool* empty) {
  *empty = true;
  if (num_rows < 0 || num_tokens < 0 || context_total < 0 || H_q < 1 || H_kv < 1 || H_q % H_kv != 0 ||
      (D != 64 && D != 128) || page_size != kPage || bt_stride < 0 || bt_len < 0 || num_pages < 0 ||
      !(scale > 0.f))
    return MS_ERR_ARG;
  const int G = H_q / H_kv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return MS_ERR_ARG;
  if (num_rows == 0 || num_tokens == 0) return MS_OK;  // no tokens: every row is a pad row
  *empty = false;
  if (!q_rot || !k_cache || !v_cache || !cu_seqlens_q || !q_start_pos || !context_lens || !block_tables || !out ||
      !workspace || num_pages < 1 || (bt_offsets == nullptr && bt_stride < 1) || (bt_offsets != nullptr && bt_len < 1))
    return MS_ERR_ARG;
  if (!aligned16(q_rot) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return MS_ERR_ARG;
  if (num_rows > kMaxRows || num_tokens > kMaxTokens) return MS_ERR_ARG;
  const WsLayout w = ws_layout(num_rows, num_tokens, context_total, H_q, H_kv, D);
  if (ws_bytes < w.total) return MS_ERR_ARG;
  const int sms = num_sms();
  if (sms <= 0) return MS_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  AttnParams& p = *params;
  p.q_rot = static_cast<const bf16*>(q_rot);
  p.cu = cu_seqlens_q;
  p.q_start = q_start_pos;
  p.ctx_lens = context_lens;
  p.bt = block_tables;
  p.bt_off = bt_offsets;
  p.bt_len = bt_offsets != nullptr ? bt_len : static_cast<int64_t>(num_rows) * bt_stride;
  p.out = static_cast<bf16*>(out);
  p.hdr = reinterpret_cast<int32_t*>(ws + w.hdr);
  p.dec_rows = reinterpret_cast<int32_t*>(ws + w.dec_rows);
  p.dec_part_base = reinterpret_cast<int32_t*>(ws + w.dec_part_base);
  p.dec_nsplit = reinterpret_cast<int32_t*>(ws + w.dec_nsplit);
  p.ch_rows = reinterpret_cast<int32_t*>(ws + w.ch_rows);
  p.dec_items = reinterpret_cast<int2*>(ws + w.dec_items);
  p.dec_cnt = reinterpret_cast<int32_t*>(ws + w.dec_cnt);
  p.ch_items = reinterpret_cast<int2*>(ws + w.ch_items);
  p.max_dec_items = w.max_dec_items;
  p.max_ch_items = w.max_ch_items;
  p.part_ml = reinterpret_cast<float*>(ws + w.part_ml);
  p.part_acc = reinterpret_cast<float*>(ws + w.part_acc);
  p.max_partials = w.max_partials;
  p.context_total = context_total;
  p.bt_stride = bt_stride;
  p.num_rows = num_rows;
  p.num_tokens = num_tokens;
  p.num_pages = num_pages;
  p.H_q = H_q;
  p.H_kv = H_kv;
  p.D = D;
  p.G = G;
  p.num_sms = sms;
  p.clear_status = clear_status ? 1 : 0;
  p.test_stall = stall_limit_ns > 0 ? 1 : 0;
  p.wait_limit_ns = stall_limit_ns > 0 ? static_cast<uint64_t>(stall_limit_ns) : 2000000000ull;
  p.scale_log2 = scale * 1.4426950408889634f;

  p.kv_q4 = nullptr;
  p.force_chunk_ctas = -1;
  p.ch_cap = 0;
  if (device_rates(&p.sm_mhz, &p.hbm_gbs, &p.l2_bytes) != MS_OK) return MS_ERR_CUDA;
  return MS_OK;
}

// The prologue as its own kernel, a programmatic dependent of the kernel
// before it: about a thread per row (one warp up to 32 rows, else at least a
// warp per scheduler).
template <bool Teams>
int launch_prologue(const AttnParams& p, cudaStream_t st) {
  if (ensure_smem_limit(prologue_kernel<Teams>, 8, prologue_words(kMaxRows) * 4) != MS_OK) return MS_ERR_CUDA;
  const int S = p.num_rows;
  const int threads = S <= 32 ? 32 : S >= 1024 ? 1024 : S <= 128 ? 128 : (S + 31) / 32 * 32;
  return launch_dependent(prologue_kernel<Teams>, dim3(1), dim3(threads), prologue_words(S) * 4, st, p) == cudaSuccess
             ? MS_OK
             : MS_ERR_CUDA;
}

}  // namespace
