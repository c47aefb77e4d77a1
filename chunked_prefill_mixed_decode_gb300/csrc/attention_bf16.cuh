// The mixed-batch attention over bf16 pools: the decode rows' phase and the set-up of
// a call, shared by the causal kernel (attention.cu) and the one of spans
// (attention_span.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attention_step.cuh"
#include "chunk_phase.cuh"
#include "mixed_step.h"
#include "ptx.cuh"

namespace {

constexpr int kChunkThreads = 32 * (4 + kSoftmaxWarps);  // warp 0 TMA + queue, 2-9 softmax, 1/10/11 MMA
// The cost model's rates (attention_step.cuh): the SM time of one 128x128 chunk
// tile, and the decode bandwidth one SM sustains, capped by HBM.
// Both SM-side rates are properties of the kernels' instruction streams, so
// they are kept per SM clock cycle and scaled by the clock the previous call
// ran at (measured on the GPU, see H_CLOCK_MHZ); HBM bandwidth comes from the
// device's memory clock and bus width.  The per-cycle figures come from
// sweeps of the split on the 8B GQA and long bimodal steps, where the kernel
// measured its clock at about 1.94 GHz (3.0 us per tile, 62 GB/s per decode
// SM); a test sweeps the split again and checks the model's choice against
// the best.
constexpr float kChunkTileCycles = 5820.f;    // SM cycles per 128x128 tile, alongside decode traffic
constexpr float kDecodeBytesPerCycle = 32.f;  // decode bytes per SM cycle at G = 1; fewer as G grows

// ----------------------------------------------------------------------------
// decode rows: split-KV, warp-level tensor-core MMAs
// ----------------------------------------------------------------------------

template <int D, int G>
struct DecCfg {
  static constexpr int NST = D == 128 ? 2 : 4;     // ring stages per warp
  static constexpr int PAGE_BYTES = kPage * D * 2;  // one page of one KV head
  static constexpr int STAGE_BYTES = 2 * PAGE_BYTES;  // K page, then V page
  static constexpr int Q_BYTES = G * D * 2;
  // per-warp tail: two Q buffers, then the ring barriers
  static constexpr int T_BAR = 2 * Q_BYTES;
  static constexpr int TAIL_BYTES = (T_BAR + NST * 8 + 127) / 128 * 128;
  // as many worker warps as the CTA has, while their rings fit in shared memory
  static constexpr int WARPS = 12 * (NST * STAGE_BYTES + TAIL_BYTES) <= 230000 ? 12 : 10;
  // all warps' stages first (each stage 1024-aligned, as 128-byte-swizzled TMA
  // tiles need), then the warps' tails
  static constexpr int TAIL_OFF = WARPS * NST * STAGE_BYTES;
  static constexpr int SMEM = TAIL_OFF + WARPS * TAIL_BYTES;
};


struct DecItem {
  int row;     // row index s
  int k;       // index among decode rows
  int hk;      // KV head
  int p0, np;  // logical pages [p0, p0 + np)
  int ctx;     // keys of the row (c + 1)
  int tok;     // packed token index of the row's query
  int part;    // partial record of query head hk * G (+ g for the others)
  int ns;      // splits of the row
  int w0;      // lane j: page id of the item's page j (its first window of 32 pages)
  int lo;      // spans: the first key that the row sees
  const int32_t* btr;  // the row's block table
};

template <bool Span>
__device__ __forceinline__ DecItem describe_dec(const AttnParams& p, int item, int split) {
  DecItem it;
  // items run (split, KV head) with the head fastest; the table has one entry per split
  const int e = item / p.H_kv;
  const int2 kl = __ldg(p.dec_items + e);  // (decode row index, split within the row)
  const int k = kl.x, sp = kl.y;
  it.hk = item - e * p.H_kv;
  it.k = k;
  it.row = __ldg(p.dec_rows + k);
  it.ctx = __ldg(p.ctx_lens + it.row);
  it.tok = __ldg(p.cu + it.row);
  const int n_pages = (it.ctx + kPage - 1) / kPage;
  it.lo = Span ? span_first(p, it.ctx - 1) : 0;
  it.p0 = (Span ? it.lo / kPage : 0) + sp * split;
  it.np = min(split, n_pages - it.p0);  // 0: a span's row without keys
  it.part = __ldg(p.dec_part_base + k) + sp * p.H_q + it.hk * p.G;
  it.ns = __ldg(p.dec_nsplit + k);
  // the first window of page ids, loaded while the item waits its turn
  const int lane = threadIdx.x & 31;
  it.btr = row_table(p, it.row);
  it.w0 = lane < it.np ? __ldg(it.btr + it.p0 + lane) : 0;
  return it;
}

// merge_splits for a KV head's G heads at once, sixteen 16-byte loads of a lane in flight: a lane looks after
// the weights of head lane % G and every (32 / G)th split, and owns D / 32 columns of every head.  (Head after
// head, two splits of eight heads took 10 us to join where their pages took 9.)  Records of splits past the
// last are those of the last with weight 0.
template <int D, int G>
__device__ __noinline__ void merge_heads(const AttnParams& p, int k, int h0, int tok, int ns, int lane) {
  constexpr int EPL = D / 32, NS = 32 / G;  // columns to a lane; splits whose weights the warp holds at a time
  constexpr int B = 16 / G;                 // splits to a batch of loads
  const int64_t base = __ldcg(p.dec_part_base + k) + h0;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + base + (lane & (G - 1));
  float M = -INFINITY;
#pragma unroll 4
  for (int j = lane / G; j < ns; j += NS) M = fmaxf(M, __ldcg(ml + static_cast<int64_t>(j) * p.H_q).x);
#pragma unroll
  for (int o = G; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float L = 0.f, out[G][EPL];
#pragma unroll
  for (int h = 0; h < G; ++h)
#pragma unroll
    for (int e = 0; e < EPL; ++e) out[h][e] = 0.f;
  for (int j0 = 0; j0 < ns; j0 += NS) {
    const int j = j0 + lane / G;
    float w = 0.f;
    if (j < ns) {
      const float2 x = __ldcg(ml + static_cast<int64_t>(j) * p.H_q);
      w = ex2(x.x - M);
      L += w * x.y;
    }
    const int nj = min(NS, ns - j0);
#pragma unroll 1
    for (int b = 0; b < nj; b += B) {
      float a[B][G][EPL];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        const float* src = p.part_acc + (base + static_cast<int64_t>(min(j0 + b + u, ns - 1)) * p.H_q) * D + lane * EPL;
#pragma unroll
        for (int h = 0; h < G; ++h) {
          if constexpr (EPL == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + h * D));
            a[u][h][0] = v.x; a[u][h][1] = v.y; a[u][h][2] = v.z; a[u][h][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(src + h * D));
            a[u][h][0] = v.x; a[u][h][1] = v.y;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < B; ++u)
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const float x = __shfl_sync(0xffffffffu, w, ((b + u) * G + h) & 31);
          const float wj = b + u < nj ? x : 0.f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) out[h][e] += wj * a[u][h][e];
        }
    }
  }
#pragma unroll
  for (int o = G; o < 32; o <<= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  bf16* dst = p.out + (static_cast<int64_t>(tok) * p.H_q + h0) * D + lane * EPL;
#pragma unroll
  for (int h = 0; h < G; ++h) {
    const float inv = 1.f / __shfl_sync(0xffffffffu, L, h);
    uint32_t x[EPL / 2];
#pragma unroll
    for (int e = 0; e < EPL; e += 2) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(out[h][e] * inv, out[h][e + 1] * inv);
      x[e / 2] = *reinterpret_cast<const uint32_t*>(&v);
    }
    if constexpr (EPL == 4) *reinterpret_cast<uint2*>(dst + h * D) = make_uint2(x[0], x[1]);
    else *reinterpret_cast<uint32_t*>(dst + h * D) = x[0];
  }
}

// Decode phase: each worker warp of the CTA (12, or 10 at D = 128, G = 8) is
// independent, with its own ring of page stages, pulling decode items until
// the queue is empty.  Per page it runs mma.sync m16n8k16 on ldmatrix
// fragments: 16 tokens against the G query heads (padded to 8).  tcgen05 does
// not fit here: its M is at least 64 rows, while a decode page is 16 rows per
// warp and a row's G query heads fill only part of N.
// Out of line, as is chunk_phase: each phase gets its own register allocation
// (inlined into one kernel body the two spill).
template <int D, int G, bool Span = false>
__device__ __noinline__ void decode_phase(const AttnParams& p, uint8_t* dsmem, const CUtensorMap* tm_k,
                                             const CUtensorMap* tm_v, const CUtensorMap* tm_kp,
                                             const CUtensorMap* tm_vp) {
  using C = DecCfg<D, G>;
  constexpr int NST = C::NST;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp >= DecCfg<D, G>::WARPS) return;  // the CTA's remaining warps have no decode slice
  uint8_t* stg = dsmem + warp * NST * C::STAGE_BYTES;             // this warp's ring stages
  uint8_t* tail = dsmem + C::TAIL_OFF + warp * C::TAIL_BYTES;     // its Q buffers and barriers
  uint64_t* full = reinterpret_cast<uint64_t*>(tail + C::T_BAR);
  const int n_items = p.hdr[H_NDEC_ITEMS];
  const int split = p.hdr[H_SPLIT];
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
  }
  __syncwarp();


  auto dequeue = [&]() -> int {
    int v = 0;
    if (lane == 0) v = atomicAdd(p.hdr + H_DEC_CTR, 1);
    return __shfl_sync(0xffffffffu, v, 0);
  };

  // issue stream: pages of `cur`, then of `nxt` (one item ahead at most)
  DecItem cur, nxt;
  int cur_id = dequeue();
  if (cur_id >= n_items) return;
  cur = describe_dec<Span>(p, cur_id, split);
  int nxt_id = dequeue();
  bool nxt_valid = nxt_id < n_items;
  if (nxt_valid) nxt = describe_dec<Span>(p, nxt_id, split);
  uint32_t seq_iss = 0, seq_con = 0;
  int iss_in_nxt = 0, iss_page = 0;
  uint32_t item_par = 0;  // q buffer of the current item
  bool failed = false;

  // lane j: page id of page (window start + j) of the issue-cursor item, and of the
  // window after it: page ids come one coalesced load per 32 pages, a window ahead
  int iss_bt = 0, iss_bt_next = 0;
  auto issue_page = [&](const DecItem& it, int pi, uint32_t qpar) {
    if ((pi & 31) == 0) {
      iss_bt = pi == 0 ? it.w0 : iss_bt_next;
      const int w = pi + 32 + lane;
      if (pi + 32 < it.np) iss_bt_next = w < it.np ? __ldg(it.btr + it.p0 + w) : 0;
    }
    int phys = __shfl_sync(0xffffffffu, iss_bt, pi & 31);
    if (lane == 0) {
      const int st = seq_iss % NST;
      uint8_t* stage = stg + st * C::STAGE_BYTES;
      if (phys < 0 || phys >= p.num_pages) {
        atomicOr(p.hdr + H_STATUS, MS_STATUS_BAD_PAGE);
        phys = 0;
      }
      const uint32_t bytes = 2 * C::PAGE_BYTES + (pi == 0 ? C::Q_BYTES : 0);
      mbar_arrive_expect_tx(full + st, bytes);
      // 16-row x 64-column slabs, 128-byte swizzled, for conflict-free ldmatrix; at
      // D = 128 each of K and V is one box of the whole page (slab 0, then slab 1)
      const int pg = phys * p.H_kv + it.hk;
      if constexpr (D == 128) {
        tma_load_4d(stage, tm_kp, 0, 0, 0, pg, full + st);
        tma_load_4d(stage + C::PAGE_BYTES, tm_vp, 0, 0, 0, pg, full + st);
      } else {
        tma_load_2d(stage, tm_k, 0, pg * kPage, full + st);
        tma_load_2d(stage + C::PAGE_BYTES, tm_v, 0, pg * kPage, full + st);
      }
      if (pi == 0)
        bulk_g2s(tail + qpar * C::Q_BYTES, p.q_rot + (static_cast<int64_t>(it.tok) * p.H_q + it.hk * G) * D,
                 C::Q_BYTES, full + st);
    }
    ++seq_iss;
  };
  auto pump = [&]() {
    while (seq_iss - seq_con < static_cast<uint32_t>(NST)) {
      if (!iss_in_nxt) {
        if (iss_page < cur.np) {
          issue_page(cur, iss_page++, item_par);
          continue;
        }
        iss_in_nxt = 1;
        iss_page = 0;
      }
      if (!nxt_valid || iss_page >= nxt.np) break;
      issue_page(nxt, iss_page++, item_par ^ 1u);
    }
  };
  pump();

  while (true) {
    // Tensor-core MMAs (mma.sync m16n8k16) on each page.  S^T = K Q^T holds
    // 16 tokens x 8 columns, a query head each (columns past G are zero, or heads again, below);
    // P^T goes back through a register transpose; O^T = V^T P^T accumulates D x 8.
    constexpr int NK = D / 16;  // 16-column steps of a K row, and 16-row blocks of O^T
    const int gq = lane >> 2, tq = lane & 3;
    // Over spans the weights are two bf16 numbers, what their rounding leaves out the second, so that of the errors only the
    // output's rounding is left.  With up to 4 heads, free columns of the product hold the heads again with those, kRest
    // columns from the weights, and O is the sum of the two (256 rows over 1024 keys, 32 / 8 heads: 2.3e-3 -> 1.7e-3 for
    // 0.3 % more time).  With 8 heads no column is free, and each fragment of V meets a second product (2.2e-3 -> 1.7e-3; 256
    // rows over 1024 keys, 64 / 8 heads: 198.9 -> 200.9 us at D = 128, 120.5 -> 120.0 at D = 64).
    constexpr int kRest = !Span || G == 8 ? 0 : G == 1 ? 1 : 4;
    constexpr bool kTwice = Span && G == 8;
    const int qh = kRest == 1 ? gq >> 1 : kRest == 4 ? gq & 3 : gq;  // head of the lane's Q words
    const int h0 = kRest == 4 ? 2 * (tq & 1) : 2 * tq, h1 = kRest == 1 ? h0 : h0 + 1;  // heads of its scores
    const float rest0 = kRest == 4 && tq >= 2 ? -1.f : 0.f, rest1 = kRest == 1 ? -1.f : rest0;
    uint32_t qb[NK][2];
    float acc[NK][4];
#pragma unroll
    for (int j = 0; j < NK; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    float mu0 = -INFINITY, mu1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads h0 and h1
    constexpr float kRescaleLog2 = 8.f;  // raise the reference max only when it grows by 2^8
    if (Span && p.sinks != nullptr && cur.p0 == cur.lo / kPage) {  // the row's first split: a key of score `sink` without a value
      if (h0 < G) mu0 = sink_log2(p, cur.hk * G + h0);
      if (h1 < G) mu1 = sink_log2(p, cur.hk * G + h1);
      if (gq == 0) {  // the lanes' sums are added up at the end
        l0 = mu0 > -INFINITY ? 1.f : 0.f;
        l1 = mu1 > -INFINITY ? 1.f : 0.f;
      }
    }
    for (int pi = 0; pi < cur.np; ++pi) {
      const int st = seq_con % NST;
      if (!mbar_wait(full + st, (seq_con / NST) & 1u, nullptr)) {
        failed = true;
        break;
      }
      const uint32_t kb = smem_u32(stg + st * C::STAGE_BYTES), vb = kb + C::PAGE_BYTES;
      if (pi == 0) {
        const uint32_t* q32 = reinterpret_cast<const uint32_t*>(tail + item_par * C::Q_BYTES);
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          qb[kk][0] = qh < G ? q32[(qh * D + 16 * kk + 2 * tq) >> 1] : 0u;
          qb[kk][1] = qh < G ? q32[(qh * D + 16 * kk + 8 + 2 * tq) >> 1] : 0u;
        }
      }
      const int tok0 = (cur.p0 + pi) * kPage;
      const int nv = min(kPage, cur.ctx - tok0);  // valid keys in this page (>= 1)
      // S^T: lane holds (token gq, columns 2 tq, 2 tq + 1: heads h0, h1) and (token gq + 8, same columns)
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        const int r = lane & 15, chunk = (kk & 3) * 2 + (lane >> 4);
        uint32_t a[4];
        ldsm_x4(kb + (kk >> 2) * 2048 + r * 128 + ((chunk ^ (r & 7)) << 4), a);
        mma_16816_bf16(c, a, qb[kk][0], qb[kk][1]);
      }
      const float sl2 = p.scale_log2;
      const int n0 = Span ? cur.lo - tok0 : 0;  // keys of the page in front of the row's span (<= 0: none)
      const bool in0 = gq < nv && (!Span || gq >= n0), in1 = gq + 8 < nv && (!Span || gq + 8 >= n0);
      const float s0 = in0 ? c[0] * sl2 : -INFINITY, s1 = in0 ? c[1] * sl2 : -INFINITY;
      const float s2 = in1 ? c[2] * sl2 : -INFINITY, s3 = in1 ? c[3] * sl2 : -INFINITY;
      float mh0 = fmaxf(s0, s2), mh1 = fmaxf(s1, s3);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mh0 = fmaxf(mh0, __shfl_xor_sync(0xffffffffu, mh0, o));
        mh1 = fmaxf(mh1, __shfl_xor_sync(0xffffffffu, mh1, o));
      }
      const bool g0 = mh0 > mu0 + kRescaleLog2, g1 = mh1 > mu1 + kRescaleLog2;
      if (__any_sync(0xffffffffu, g0 || g1)) {
        const float m0 = g0 ? mh0 : mu0, m1 = g1 ? mh1 : mu1;
        const float a0 = g0 ? ex2(mu0 - m0) : 1.f, a1 = g1 ? ex2(mu1 - m1) : 1.f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          acc[j][0] *= a0;
          acc[j][1] *= a1;
          acc[j][2] *= a0;
          acc[j][3] *= a1;
        }
        l0 *= a0;
        l1 *= a1;
        mu0 = m0;
        mu1 = m1;
      }
      const float p0 = ex2(s0 - mu0), p1 = ex2(s1 - mu1), p2 = ex2(s2 - mu0), p3 = ex2(s3 - mu1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      __nv_bfloat162 h01 = __floats2bfloat162_rn(p0, p1), h23 = __floats2bfloat162_rn(p2, p3);
      if constexpr (kRest > 0) {
        const float2 f01 = __bfloat1622float2(h01), f23 = __bfloat1622float2(h23);
        h01 = __floats2bfloat162_rn(fmaf(rest0, f01.x, p0), fmaf(rest1, f01.y, p1));
        h23 = __floats2bfloat162_rn(fmaf(rest0, f23.x, p2), fmaf(rest1, f23.y, p3));
      }
      // P^T as the B operand: lane holds (tokens 2 tq, 2 tq + 1 | + 8, column gq)
      const uint32_t b0 = movmatrix_trans(*reinterpret_cast<uint32_t*>(&h01));
      const uint32_t b1 = movmatrix_trans(*reinterpret_cast<uint32_t*>(&h23));
      uint32_t r0 = 0, r1 = 0;
      if constexpr (kTwice) {  // what the rounding of the weights leaves out
        const float2 f01 = __bfloat1622float2(h01), f23 = __bfloat1622float2(h23);
        const __nv_bfloat162 e01 = __floats2bfloat162_rn(p0 - f01.x, p1 - f01.y), e23 = __floats2bfloat162_rn(p2 - f23.x, p3 - f23.y);
        r0 = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&e01));
        r1 = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&e23));
      }
      if (nv < kPage) {
        // rows past the context in the last page may hold stale (even non-finite) data:
        // zero them in V so that P = 0 times V stays 0
        uint8_t* v0 = stg + st * C::STAGE_BYTES + C::PAGE_BYTES;
        for (int i = lane; i < (kPage - nv) * (D / 8); i += 32) {
          const int r = nv + i / (D / 8), cc = i % (D / 8);  // row, 16-byte chunk of the row
          *reinterpret_cast<uint4*>(v0 + (cc >> 3) * 2048 + r * 128 + (cc & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // ordered before the next copy into this stage
        __syncwarp();
      }
      if (Span && n0 > 0) {  // so may those in front of the span, in its first page
        uint8_t* v0 = stg + st * C::STAGE_BYTES + C::PAGE_BYTES;
        for (int i = lane; i < n0 * (D / 8); i += 32) {
          const int r = i / (D / 8), cc = i % (D / 8);
          *reinterpret_cast<uint4*>(v0 + (cc >> 3) * 2048 + r * 128 + (cc & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        const int r = ((lane >> 4) << 3) + (lane & 7), chunk = (j & 3) * 2 + ((lane >> 3) & 1);
        uint32_t a[4];
        ldsm_x4_trans(vb + (j >> 2) * 2048 + r * 128 + ((chunk ^ (r & 7)) << 4), a);
        mma_16816_bf16(acc[j], a, b0, b1);
        if constexpr (kTwice) mma_16816_bf16(acc[j], a, r0, r1);
      }
      __syncwarp();
      ++seq_con;
      pump();
    }
    if (failed) break;
    if constexpr (kRest > 0) {
#pragma unroll
      for (int j = 0; j < NK; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (kRest == 4) acc[j][e] += __shfl_xor_sync(0xffffffffu, acc[j][e], 2);
          else if (e % 2 == 0) acc[j][e] += acc[j][e + 1];
        }
    }
    // O^T: lane holds (d 16 j + gq, columns 2 tq, 2 tq + 1) and (d 16 j + gq + 8, same columns); column g < G is head g
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hh = 2 * tq + e;
      if (hh >= G) continue;
      const float L = e == 0 ? l0 : l1, M = e == 0 ? mu0 : mu1;
      if (cur.ns == 1) {
        const float inv = !Span || L > 0.f ? 1.f / L : 0.f;  // no key at all: zeros
        bf16* dst = p.out + (static_cast<int64_t>(cur.tok) * p.H_q + cur.hk * G + hh) * D;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          dst[16 * j + gq] = __float2bfloat16_rn(acc[j][e] * inv);
          dst[16 * j + gq + 8] = __float2bfloat16_rn(acc[j][2 + e] * inv);
        }
      } else {
        const int64_t rec = cur.part + hh;
        float* dst = p.part_acc + rec * D;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          dst[16 * j + gq] = acc[j][e];
          dst[16 * j + gq + 8] = acc[j][2 + e];
        }
        if (gq == 0) *reinterpret_cast<float2*>(p.part_ml + rec * 2) = make_float2(M, L);
      }
    }
    if (cur.ns > 1) {
      __threadfence();  // this split's records are visible before it is counted
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atomicAdd(p.dec_cnt + cur.k * p.H_kv + cur.hk, 1) == cur.ns - 1;
      last = __shfl_sync(0xffffffffu, last, 0);
      if (last) {
        __threadfence();
        if constexpr (Span) merge_heads<D, G>(p, cur.k, cur.hk * G, cur.tok, cur.ns, lane);
        else merge_splits<D>(p, cur.k, cur.hk * G, G, cur.tok, cur.ns, lane);
      }
    }
    if (!nxt_valid) break;
    // advance: the next item becomes current; dequeue one more
    cur = nxt;
    item_par ^= 1u;
    iss_in_nxt = 0;  // the issue cursor (iss_page) already points into the new current item
    nxt_id = dequeue();
    nxt_valid = nxt_id < n_items;
    if (nxt_valid) nxt = describe_dec<Span>(p, nxt_id, split);
    pump();
  }
  if (failed) {
    if (lane == 0) atomicOr(p.hdr + H_STATUS, MS_STATUS_TIMEOUT);
    // let copies already in flight land before the CTA's shared memory is released
    while (seq_con < seq_iss) {
      mbar_wait(full + seq_con % NST, (seq_con / NST) & 1u, nullptr, 200000000ull);
      ++seq_con;
    }
  }
}

static_assert(DecCfg<128, 8>::SMEM <= 232448 && DecCfg<64, 8>::SMEM <= 232448 && DecCfg<128, 4>::WARPS == 12,
              "decode rings exceed the per-CTA shared-memory limit");

// barriers of one finished phase, invalidated before the memory is reused
template <int D, int G>
__device__ __forceinline__ void invalidate_phase_barriers(uint8_t* smem, bool chunk) {
  if (chunk) {
    if (threadIdx.x == 0) {
      ChBars* bars = reinterpret_cast<ChBars*>(smem + ChCfg<D>::BAR_OFF);
      uint64_t* b0 = &bars->q_full;
      uint64_t* b1 = &bars->mma_done[2];
      for (uint64_t* b = b0; b <= b1; ++b) mbar_inval(b);
    }
  } else if ((threadIdx.x & 31) == 0 && (threadIdx.x >> 5) < DecCfg<D, G>::WARPS) {
    using C = DecCfg<D, G>;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::TAIL_OFF + (threadIdx.x >> 5) * C::TAIL_BYTES + C::T_BAR);
    for (int i = 0; i < C::NST; ++i) mbar_inval(full + i);
  }
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------

// decode worker warps per CTA for head dim D and group size G
int dec_warps(int D, int G) {
  switch (D * 100 + G) {
    case 6401: return DecCfg<64, 1>::WARPS;
    case 6402: return DecCfg<64, 2>::WARPS;
    case 6404: return DecCfg<64, 4>::WARPS;
    case 6408: return DecCfg<64, 8>::WARPS;
    case 12801: return DecCfg<128, 1>::WARPS;
    case 12802: return DecCfg<128, 2>::WARPS;
    case 12804: return DecCfg<128, 4>::WARPS;
    default: return DecCfg<128, 8>::WARPS;
  }
}

// An attention call's launch parameters: the kernels' arguments and the four
// tensor maps.
struct AttnPlan {
  AttnParams p;
  CUtensorMap tq, tk, tv, tvp, tkp;
};

// step_setup for the bf16 pools, and their tensor maps.
int attention_setup(const void* q_rot, const void* k_cache, const void* v_cache, int32_t num_pages,
                    const int32_t* cu_seqlens_q, const int32_t* q_start_pos, const int32_t* context_lens,
                    const int32_t* block_tables, const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride,
                    int32_t num_rows, int32_t num_tokens, int64_t context_total, int32_t H_q, int32_t H_kv,
                    int32_t D, int32_t page_size, float scale, void* out, void* workspace, size_t ws_bytes,
                    bool clear_status, int64_t stall_limit_ns, AttnPlan* L, bool* empty) {
  const int rc = step_setup(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables,
                            bt_offsets, bt_len, bt_stride, num_rows, num_tokens, context_total, H_q, H_kv, D, page_size,
                            scale, out, workspace, ws_bytes, clear_status, stall_limit_ns, &L->p, empty);
  if (rc != MS_OK || *empty) return rc;
  AttnParams& p = L->p;
  const int G = p.G;
  p.dec_workers = p.num_sms * dec_warps(D, G);
  p.tile_cycles = kChunkTileCycles;
  p.dec_bytes_cycle = kDecodeBytesPerCycle / (1.f + 0.18f * (G - 1));
  p.key_bytes = 4.f * D;
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return MS_ERR_CUDA;

  CUtensorMap& tq = L->tq;
  CUtensorMap& tk = L->tk;
  CUtensorMap& tv = L->tv;
  CUtensorMap& tvp = L->tvp;
  CUtensorMap& tkp = L->tkp;
  {
    const cuuint64_t dq[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H_q),
                              static_cast<cuuint64_t>(num_tokens)};
    const cuuint64_t sq[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H_q) * D * 2};
    const cuuint32_t bq[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(128 / G)};
    const cuuint64_t dk[2] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(num_pages) * H_kv * kPage};
    const cuuint64_t sk[1] = {static_cast<cuuint64_t>(D) * 2};
    const cuuint32_t bk[2] = {64, static_cast<cuuint32_t>(kPage)};
    if (!encode_bf16(enc, &tq, q_rot, 3, dq, sq, bq) || !encode_bf16(enc, &tk, k_cache, 2, dk, sk, bk) ||
        !encode_bf16(enc, &tv, v_cache, 2, dk, sk, bk))
      return MS_ERR_ARG;
    tvp = tv;  // at D = 64 a page is one 2 KB box of tv (and of tk)
    tkp = tk;
    if (D == 128) {
      // K and V by whole pages (V for the chunk tiles, both for the decode ring):
      // (64 columns, 16 rows, 2 slabs, page x KV head), so that one box lands as
      // the page's slab 0 then its slab 1
      const cuuint64_t dv[4] = {64, static_cast<cuuint64_t>(kPage), 2,
                                static_cast<cuuint64_t>(num_pages) * H_kv};
      const cuuint64_t sv[3] = {static_cast<cuuint64_t>(D) * 2, 128,
                                static_cast<cuuint64_t>(kPage) * D * 2};
      const cuuint32_t bv[4] = {64, static_cast<cuuint32_t>(kPage), 2, 1};
      if (!encode_bf16(enc, &tvp, v_cache, 4, dv, sv, bv) || !encode_bf16(enc, &tkp, k_cache, 4, dv, sv, bv))
        return MS_ERR_ARG;
    }
  }
  return MS_OK;
}

}  // namespace
