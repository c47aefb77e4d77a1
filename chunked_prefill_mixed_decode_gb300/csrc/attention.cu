// Mixed-batch attention over a paged KV cache, sm_103a.
//
// A step packs single-token decodes next to prefill chunks ("Chunked Prefill:
// Ending the Great Stall", sections 03-04).  Row s has d_s new tokens at
// absolute positions [c_s, c_s + d_s); its query at position p attends keys
// 0..p ("Chunked Prefill 的 Token 预算" (zwjcode.cn), sections 02 and 07):
// the cached prefix [0, c) plus its own chunk causally.  The two row kinds sit
// on opposite sides of the roofline ("Chunked Prefill: Ending the Great
// Stall", section 03; "Splitting Prefill From Decode Inside a Step", "Two
// kernels with different limiting resources"), so they take two paths:
//
//   decode rows (d = 1): split-KV with warp-level tensor-core MMAs.  One warp
//     owns a work item (row, KV head, span of pages) and streams its pages
//     through a private ring in shared memory with TMA (128-byte swizzled
//     16-row boxes); the G query heads of the KV head share every page read.
//     Per page, S^T = K Q^T (16 tokens x G heads, padded to 8) and
//     O^T += V^T P^T run as mma.sync m16n8k16 on ldmatrix fragments, with P
//     transposed in registers.  Each item leaves a partial (max, sum,
//     accumulator); the last split of a (row, KV head) to finish merges them.
//   chunk rows (d > 1): tcgen05 tensor cores.  A work item is a pair of
//     128-row query tiles (128/G tokens x G heads of one KV head each) that
//     walk 64-key tiles of the prefix and their own chunk together.  TMA loads
//     Q and K pages (one 16-row box per page and 64-column slab, 128-byte
//     swizzle) and V pages (one box per page, both slabs, at D = 128); S = Q K^T
//     lands in TMEM; two groups of four softmax warps, one
//     per query tile and one row per thread, write P (bf16) back over S, and
//     O += P V runs with P as the TMEM operand, accumulating in TMEM and
//     rescaled only when a row's maximum grows by more than a factor 2^8.
//
// A one-CTA prologue validates the metadata, chooses the split size, orders
// rows longest-first, expands the per-row item counts into flat item tables
// and decides how many CTAs start on chunk tiles.  One persistent kernel (a
// CTA per SM) then runs both queues: CTAs on SMs below the split start on
// chunk tiles, the rest on decode items, and each moves to the other queue
// when its own runs dry.  Work comes from atomic counters; no CTA waits on
// another.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "append_rope.cuh"
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

// The append and the prologue as one kernel (the step call on small steps):
// CTA 0 runs the prologue, the others the append's work units.  Launched in
// plain stream order, so nothing of the step before is still running.
template <typename Idx>
__global__ void __launch_bounds__(kAppendThreads) append_prologue_kernel(AppendArgs a, AttnParams p) {
  griddep_launch_dependents();  // the attention kernel may start its set-up
  if (blockIdx.x == 0) {
    prologue_body<false>(p);
    return;
  }
  append_rope_units<Idx>(a, static_cast<Idx>(blockIdx.x - 1) * kAppendThreads + threadIdx.x,
                         static_cast<Idx>(gridDim.x - 1) * kAppendThreads);
}

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
  const int32_t* btr;  // the row's block table
};

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
  it.p0 = sp * split;
  it.np = min(split, n_pages - it.p0);
  it.part = __ldg(p.dec_part_base + k) + sp * p.H_q + it.hk * p.G;
  it.ns = __ldg(p.dec_nsplit + k);
  // the first window of page ids, loaded while the item waits its turn
  const int lane = threadIdx.x & 31;
  it.btr = row_table(p, it.row);
  it.w0 = lane < it.np ? __ldg(it.btr + it.p0 + lane) : 0;
  return it;
}


// Decode phase: each worker warp of the CTA (12, or 10 at D = 128, G = 8) is
// independent, with its own ring of page stages, pulling decode items until
// the queue is empty.  Per page it runs mma.sync m16n8k16 on ldmatrix
// fragments: 16 tokens against the G query heads (padded to 8).  tcgen05 does
// not fit here: its M is at least 64 rows, while a decode page is 16 rows per
// warp and a row's G query heads fill only part of N.

// Out of line, as is chunk_phase: each phase gets its own register allocation
// (inlined into one kernel body the two spill).
template <int D, int G>
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
  cur = describe_dec(p, cur_id, split);
  int nxt_id = dequeue();
  bool nxt_valid = nxt_id < n_items;
  if (nxt_valid) nxt = describe_dec(p, nxt_id, split);
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
    // 16 tokens x 8 query heads (heads past G are zero); P^T goes back through
    // a register transpose; O^T = V^T P^T accumulates D x 8.
    constexpr int NK = D / 16;  // 16-column steps of a K row, and 16-row blocks of O^T
    const int gq = lane >> 2, tq = lane & 3;
    uint32_t qb[NK][2];
    float acc[NK][4];
#pragma unroll
    for (int j = 0; j < NK; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    float mu0 = -INFINITY, mu1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2 tq and 2 tq + 1
    constexpr float kRescaleLog2 = 8.f;  // raise the reference max only when it grows by 2^8
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
          qb[kk][0] = gq < G ? q32[(gq * D + 16 * kk + 2 * tq) >> 1] : 0u;
          qb[kk][1] = gq < G ? q32[(gq * D + 16 * kk + 8 + 2 * tq) >> 1] : 0u;
        }
      }
      const int tok0 = (cur.p0 + pi) * kPage;
      const int nv = min(kPage, cur.ctx - tok0);  // valid keys in this page (>= 1)
      // S^T: lane holds (token gq, heads 2 tq, 2 tq + 1) and (token gq + 8, same heads)
      float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        const int r = lane & 15, chunk = (kk & 3) * 2 + (lane >> 4);
        uint32_t a[4];
        ldsm_x4(kb + (kk >> 2) * 2048 + r * 128 + ((chunk ^ (r & 7)) << 4), a);
        mma_16816_bf16(c, a, qb[kk][0], qb[kk][1]);
      }
      const float sl2 = p.scale_log2;
      const float s0 = gq < nv ? c[0] * sl2 : -INFINITY, s1 = gq < nv ? c[1] * sl2 : -INFINITY;
      const float s2 = gq + 8 < nv ? c[2] * sl2 : -INFINITY, s3 = gq + 8 < nv ? c[3] * sl2 : -INFINITY;
      float mh0 = fmaxf(s0, s2), mh1 = fmaxf(s1, s3);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mh0 = fmaxf(mh0, __shfl_xor_sync(0xffffffffu, mh0, o));
        mh1 = fmaxf(mh1, __shfl_xor_sync(0xffffffffu, mh1, o));
      }
      const bool g0 = mh0 > mu0 + kRescaleLog2, g1 = mh1 > mu1 + kRescaleLog2;
      if (__any_sync(0xffffffffu, g0 || g1)) {
        const float n0 = g0 ? mh0 : mu0, n1 = g1 ? mh1 : mu1;
        const float a0 = g0 ? ex2(mu0 - n0) : 1.f, a1 = g1 ? ex2(mu1 - n1) : 1.f;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          acc[j][0] *= a0;
          acc[j][1] *= a1;
          acc[j][2] *= a0;
          acc[j][3] *= a1;
        }
        l0 *= a0;
        l1 *= a1;
        mu0 = n0;
        mu1 = n1;
      }
      const float p0 = ex2(s0 - mu0), p1 = ex2(s1 - mu1), p2 = ex2(s2 - mu0), p3 = ex2(s3 - mu1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      __nv_bfloat162 h01 = __floats2bfloat162_rn(p0, p1), h23 = __floats2bfloat162_rn(p2, p3);
      // P^T as the B operand: lane holds (tokens 2 tq, 2 tq + 1 | + 8, head gq)
      const uint32_t b0 = movmatrix_trans(*reinterpret_cast<uint32_t*>(&h01));
      const uint32_t b1 = movmatrix_trans(*reinterpret_cast<uint32_t*>(&h23));
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
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        const int r = ((lane >> 4) << 3) + (lane & 7), chunk = (j & 3) * 2 + ((lane >> 3) & 1);
        uint32_t a[4];
        ldsm_x4_trans(vb + (j >> 2) * 2048 + r * 128 + ((chunk ^ (r & 7)) << 4), a);
        mma_16816_bf16(acc[j], a, b0, b1);
      }
      __syncwarp();
      ++seq_con;
      pump();
    }
    if (failed) break;
    // O^T: lane holds (d 16 j + gq, heads 2 tq, 2 tq + 1) and (d 16 j + gq + 8, same heads)
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
        const float inv = 1.f / L;
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
        merge_splits<D>(p, cur.k, cur.hk * G, G, cur.tok, cur.ns, lane);
      }
    }
    if (!nxt_valid) break;
    // advance: the next item becomes current; dequeue one more
    cur = nxt;
    item_par ^= 1u;
    iss_in_nxt = 0;  // the issue cursor (iss_page) already points into the new current item
    nxt_id = dequeue();
    nxt_valid = nxt_id < n_items;
    if (nxt_valid) nxt = describe_dec(p, nxt_id, split);
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

// One persistent CTA per SM.  CTAs on SMs below hdr[H_CHUNK_CTAS] start on chunk
// tiles (tensor cores), the others on decode items (HBM), so the two kinds of
// work run side by side; a CTA whose queue runs dry moves to the other queue.
template <int D, int G>
__global__ void __launch_bounds__(kChunkThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_vp,
                     const __grid_constant__ CUtensorMap tm_kp,
                     AttnParams p) {
  // no static shared memory: the dynamic block starts 1024-aligned, as the
  // 128-byte-swizzled TMA tiles and MMA descriptors require
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  if ((smem_u32(smem) & 1023u) != 0) {
    griddep_wait();
    if (threadIdx.x == 0) atomicOr(p.hdr + H_STATUS, MS_STATUS_INTERNAL);
    return;
  }
  // set-up that needs nothing from the kernels before: it overlaps their tail
  // when this kernel is launched as a programmatic dependent
  uint32_t* tmem_slot = &reinterpret_cast<ChBars*>(smem + ChCfg<D>::BAR_OFF)->tmem;
  if (warp == 1) {
    tmem_alloc(tmem_slot, ChCfg<D>::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();  // the prologue's item tables (and, through it, the append's q_rot and pages)
  // CTA 0 times its own run in SM cycles and in ns: the SM clock, for the next call's cost model
  const long long clk0 = clock64();
  const uint64_t ns0 = globaltimer_ns();
  const int n_ch_items = p.hdr[H_NCH_ITEMS];
  const int n_dec_items = p.hdr[H_NDEC_ITEMS];
  __syncthreads();  // every thread holds the address before the phases reuse the memory
  if (n_ch_items == 0 && n_dec_items == 0) {
    if (warp == 1) tmem_dealloc(tmem, ChCfg<D>::TMEM_COLS);
    return;
  }
  // Which CTAs start on chunk work goes by the SM they run on, not by block
  // index: as a programmatic dependent, the kernel's blocks reach SMs in an
  // order set by the kernels still draining, and a split by block index then
  // lands differently from step to step (up to 6 % slower on the long bimodal
  // step).  It only sets where a CTA starts; any count of chunk-first CTAs is
  // correct, since a CTA whose queue runs dry takes the other one.
  uint32_t smid;
  asm volatile("mov.u32 %0, %%smid;" : "=r"(smid));
  const bool chunk_first = static_cast<int>(smid) < p.hdr[H_CHUNK_CTAS];
  for (int ph = 0; ph < 2; ++ph) {
    const bool chunk = (ph == 0) == chunk_first;
    if (chunk && n_ch_items > 0) {
      chunk_phase<D, G>(&tm_q, &tm_k, &tm_v, &tm_vp, p, smem, tmem);
      tc_fence_before();
      __syncthreads();
      const bool aborted = reinterpret_cast<ChBars*>(smem + ChCfg<D>::BAR_OFF)->abort != 0;
      invalidate_phase_barriers<D, G>(smem, true);
      __syncthreads();
      if (aborted) break;
    } else if (!chunk && n_dec_items > 0) {
      decode_phase<D, G>(p, smem, &tm_k, &tm_v, &tm_kp, &tm_vp);
      __syncwarp();
      invalidate_phase_barriers<D, G>(smem, false);
      __syncthreads();
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, ChCfg<D>::TMEM_COLS);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const uint64_t ns = globaltimer_ns() - ns0;
    if (ns >= 20000)  // long enough for the timer's resolution
      p.hdr[H_CLOCK_MHZ] = static_cast<int>(static_cast<double>(clock64() - clk0) * 1e3 / static_cast<double>(ns));
  }
}


}  // namespace

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------

namespace {

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

template <int D, int G>
int launch_paths(const AttnParams& p, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                 const CUtensorMap& tvp, const CUtensorMap& tkp, int n_ctas, cudaStream_t st) {
  constexpr int smem = ChCfg<D>::SMEM > DecCfg<D, G>::SMEM ? ChCfg<D>::SMEM : DecCfg<D, G>::SMEM;
  static_assert(smem <= 232448, "attention kernel exceeds the per-CTA shared-memory limit");
  const int slot = (D == 128 ? 4 : 0) + (G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3);  // one bit per instance
  if (ensure_smem_limit(attention_kernel<D, G>, slot, smem) != MS_OK) return MS_ERR_CUDA;
  if (launch_dependent(attention_kernel<D, G>, dim3(n_ctas), dim3(kChunkThreads), smem, st, tq, tk, tv, tvp, tkp,
                       p) != cudaSuccess)
    return MS_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}

}  // namespace

extern "C" MS_API size_t ms_attention_workspace_size(int32_t max_rows, int32_t max_tokens, int64_t max_context_total,
                                                     int32_t H_q, int32_t H_kv, int32_t D) {
  if (max_rows < 0 || max_tokens < 0 || max_context_total < 0 || H_q < 1 || H_kv < 1 || H_q % H_kv != 0 ||
      (D != 64 && D != 128))
    return 0;
  return ws_layout(max_rows, max_tokens, max_context_total, H_q, H_kv, D).total;
}

extern "C" MS_API int ms_cost_model_rates(float* sm_mhz, float* hbm_gbs) {
  if (sm_mhz == nullptr || hbm_gbs == nullptr) return MS_ERR_ARG;
  float l2 = 0.f;
  return device_rates(sm_mhz, hbm_gbs, &l2);
}

extern "C" MS_API int ms_num_sms(void) {
  const int n = num_sms();
  return n > 0 ? n : MS_ERR_CUDA;
}

namespace {

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

// The persistent attention kernel for the call's head dim and group size.
int launch_attention(const AttnPlan& L, cudaStream_t st) {
  const AttnParams& p = L.p;
  const CUtensorMap &tq = L.tq, &tk = L.tk, &tv = L.tv, &tvp = L.tvp, &tkp = L.tkp;
  const int n_ctas = p.num_sms;  // one persistent CTA per SM
  int rc = MS_ERR_ARG;
  switch (p.D * 100 + p.G) {
    case 6401: rc = launch_paths<64, 1>(p, tq, tk, tv, tvp, tkp, n_ctas, st); break;
    case 6402: rc = launch_paths<64, 2>(p, tq, tk, tv, tvp, tkp, n_ctas, st); break;
    case 6404: rc = launch_paths<64, 4>(p, tq, tk, tv, tvp, tkp, n_ctas, st); break;
    case 6408: rc = launch_paths<64, 8>(p, tq, tk, tv, tvp, tkp, n_ctas, st); break;
    case 12801: rc = launch_paths<128, 1>(p, tq, tk, tv, tvp, tkp, n_ctas, st); break;
    case 12802: rc = launch_paths<128, 2>(p, tq, tk, tv, tvp, tkp, n_ctas, st); break;
    case 12804: rc = launch_paths<128, 4>(p, tq, tk, tv, tvp, tkp, n_ctas, st); break;
    case 12808: rc = launch_paths<128, 8>(p, tq, tk, tv, tvp, tkp, n_ctas, st); break;
    default: break;
  }
  return rc;
}

// The attention call behind the attention entry points: prologue, then the
// persistent kernel.  Every argument check comes before the first enqueue, so
// a call that returns an error has put nothing on the stream.  *launched tells
// whether kernels were enqueued (a step with no tokens enqueues none).
int attention_call(const void* q_rot, const void* k_cache, const void* v_cache, int32_t num_pages,
                   const int32_t* cu_seqlens_q, const int32_t* q_start_pos, const int32_t* context_lens,
                   const int32_t* block_tables, const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride,
                   int32_t num_rows, int32_t num_tokens,
                   int64_t context_total, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size, float scale,
                   void* out, void* workspace, size_t ws_bytes, ms_stream_t stream, bool clear_status,
                   int64_t stall_limit_ns, bool* launched, int32_t force_chunk_ctas = -1) {
  *launched = false;
  AttnPlan L;
  bool empty = true;
  const int rc = attention_setup(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens,
                                 block_tables, bt_offsets, bt_len, bt_stride, num_rows, num_tokens, context_total, H_q,
                                 H_kv, D, page_size, scale, out, workspace, ws_bytes, clear_status, stall_limit_ns, &L,
                                 &empty);
  if (rc != MS_OK || empty) return rc;
  L.p.force_chunk_ctas = force_chunk_ctas;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  *launched = true;  // from here on, kernels may be on the stream
  const int rp = launch_prologue<false>(L.p, st);
  return rp != MS_OK ? rp : launch_attention(L, st);
}

// Steps of at most this many rows run the prologue inside the append's launch
// (its shared memory, prologue_words(rows), then sits on every append CTA:
// 20 KB at this bound, under an eighth of the SM's for 8 resident CTAs).
constexpr int kFuseRows = 1024;

}  // namespace

extern "C" MS_API int ms_mixed_step_attention(const void* q_rot, const void* k_cache, const void* v_cache,
                                              int32_t num_pages, const int32_t* cu_seqlens_q,
                                              const int32_t* q_start_pos, const int32_t* context_lens,
                                              const int32_t* block_tables, int32_t bt_stride, int32_t num_rows,
                                              int32_t num_tokens, int64_t context_total, int32_t H_q, int32_t H_kv,
                                              int32_t D, int32_t page_size, float scale, void* out, void* workspace,
                                              size_t ws_bytes, ms_stream_t stream) {
  bool launched = false;
  return attention_call(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables,
                        nullptr, 0, bt_stride, num_rows, num_tokens, context_total, H_q, H_kv, D, page_size, scale, out,
                        workspace, ws_bytes, stream, false, 0, &launched);
}

extern "C" MS_API int ms_mixed_step_attention_ragged(const void* q_rot, const void* k_cache, const void* v_cache,
                                                     int32_t num_pages, const int32_t* cu_seqlens_q,
                                                     const int32_t* q_start_pos, const int32_t* context_lens,
                                                     const int32_t* bt_offsets, const int32_t* bt_pages,
                                                     int64_t num_bt_pages, int32_t num_rows, int32_t num_tokens,
                                                     int64_t context_total, int32_t H_q, int32_t H_kv, int32_t D,
                                                     int32_t page_size, float scale, void* out, void* workspace,
                                                     size_t ws_bytes, ms_stream_t stream) {
  if (bt_offsets == nullptr && num_rows > 0 && num_tokens > 0) return MS_ERR_ARG;
  bool launched = false;
  return attention_call(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, bt_pages,
                        bt_offsets, num_bt_pages, 0, num_rows, num_tokens, context_total, H_q, H_kv, D, page_size,
                        scale, out, workspace, ws_bytes, stream, false, 0, &launched);
}

extern "C" MS_API int ms_mixed_step(const void* q, const void* k, const void* v, const int32_t* positions,
                                   const int32_t* slot_mapping, const float* cos_tab, const float* sin_tab,
                                   int32_t max_pos, void* k_cache, void* v_cache, int32_t num_pages, void* q_rot,
                                   const int32_t* cu_seqlens_q, const int32_t* q_start_pos,
                                   const int32_t* context_lens, const int32_t* block_tables,
                                   const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride, int32_t num_rows,
                                   int32_t num_tokens, int64_t context_total, int32_t H_q, int32_t H_kv, int32_t D,
                                   int32_t page_size, float scale, void* out, void* workspace, size_t ws_bytes,
                                   int32_t* dev_status, ms_stream_t stream) {
  AppendArgs a;
  int64_t units = 0;
  int rc = append_setup(q, k, v, positions, slot_mapping, num_tokens, cos_tab, sin_tab, max_pos, k_cache, v_cache,
                        num_pages, q_rot, H_q, H_kv, D, page_size, dev_status, &a, &units);
  if (rc != MS_OK) return rc;
  AttnPlan L;
  bool empty = true;
  rc = attention_setup(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables,
                       bt_offsets, bt_offsets != nullptr ? bt_len : 0, bt_offsets != nullptr ? 0 : bt_stride, num_rows,
                       num_tokens, context_total, H_q, H_kv, D, page_size, scale, out, workspace, ws_bytes, false, 0,
                       &L, &empty);
  if (rc != MS_OK) return rc;
  if (units == 0) return MS_OK;  // no tokens: nothing to append or attend
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (empty || num_rows > kFuseRows) {
    rc = ms_kv_append_rope(q, k, v, positions, slot_mapping, num_tokens, cos_tab, sin_tab, max_pos, k_cache, v_cache,
                           num_pages, q_rot, H_q, H_kv, D, page_size, dev_status, stream);
    if (rc != MS_OK || empty) return rc;
    rc = launch_prologue<false>(L.p, st);
    return rc != MS_OK ? rc : launch_attention(L, st);
  }
  // CTA 0 runs the prologue beside the append's CTAs; plain stream order, so the
  // step before has finished with the workspace
  const int64_t blocks = 1 + append_blocks(units, L.p.num_sms);
  const int smem = prologue_words(num_rows) * 4;
  if (units + blocks * kAppendThreads < (int64_t{1} << 31)) {
    if (ensure_smem_limit(append_prologue_kernel<uint32_t>, 9, prologue_words(kFuseRows) * 4) != MS_OK)
      return MS_ERR_CUDA;
    append_prologue_kernel<uint32_t><<<static_cast<unsigned>(blocks), kAppendThreads, smem, st>>>(a, L.p);
  } else {
    if (ensure_smem_limit(append_prologue_kernel<int64_t>, 10, prologue_words(kFuseRows) * 4) != MS_OK)
      return MS_ERR_CUDA;
    append_prologue_kernel<int64_t><<<static_cast<unsigned>(blocks), kAppendThreads, smem, st>>>(a, L.p);
  }
  if (cudaGetLastError() != cudaSuccess) return MS_ERR_CUDA;
  return launch_attention(L, st);
}

extern "C" MS_API int ms_test_attention_stall(const void* q_rot, const void* k_cache, const void* v_cache,
                                              int32_t num_pages, const int32_t* cu_seqlens_q,
                                              const int32_t* q_start_pos, const int32_t* context_lens,
                                              const int32_t* block_tables, int32_t bt_stride, int32_t num_rows,
                                              int32_t num_tokens, int64_t context_total, int32_t H_q, int32_t H_kv,
                                              int32_t D, int32_t page_size, float scale, void* out, void* workspace,
                                              size_t ws_bytes, int64_t wait_limit_ns, ms_stream_t stream) {
  if (wait_limit_ns < 100000 || wait_limit_ns > 2000000000ll) return MS_ERR_ARG;  // 0.1 ms .. 2 s
  bool launched = false;
  return attention_call(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables,
                        nullptr, 0, bt_stride, num_rows, num_tokens, context_total, H_q, H_kv, D, page_size, scale, out,
                        workspace, ws_bytes, stream, false, wait_limit_ns, &launched);
}

extern "C" MS_API int ms_test_attention_split(const void* q_rot, const void* k_cache, const void* v_cache,
                                              int32_t num_pages, const int32_t* cu_seqlens_q,
                                              const int32_t* q_start_pos, const int32_t* context_lens,
                                              const int32_t* block_tables, const int32_t* bt_offsets, int64_t bt_len,
                                              int32_t bt_stride, int32_t num_rows, int32_t num_tokens,
                                              int64_t context_total, int32_t H_q, int32_t H_kv, int32_t D,
                                              int32_t page_size, float scale, void* out, void* workspace,
                                              size_t ws_bytes, int32_t chunk_ctas, ms_stream_t stream) {
  if (chunk_ctas < 0) return MS_ERR_ARG;
  bool launched = false;
  return attention_call(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables,
                        bt_offsets, bt_offsets != nullptr ? bt_len : 0, bt_offsets != nullptr ? 0 : bt_stride,
                        num_rows, num_tokens, context_total, H_q, H_kv, D, page_size, scale, out, workspace, ws_bytes,
                        stream, false, 0, &launched, chunk_ctas);
}

extern "C" MS_API int ms_read_status(int32_t* dev_status, ms_stream_t stream, int32_t* host_status) {
  if (dev_status == nullptr || host_status == nullptr) return MS_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, dev_status, sizeof(v), cudaMemcpyDeviceToHost, st) != cudaSuccess) return MS_ERR_CUDA;
  if (cudaMemsetAsync(dev_status, 0, sizeof(int32_t), st) != cudaSuccess) return MS_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MS_ERR_CUDA;
  *host_status = v;
  return v == 0 ? MS_OK : MS_ERR_DEVICE;
}

// ----------------------------------------------------------------------------
// attention without a caller workspace
// ----------------------------------------------------------------------------
//
// Some callers cannot hand the library a workspace: a serving process that
// reserves nearly all device memory for its KV-cache pool at start-up and
// leaves nothing for a second allocator, or host code that must not call
// cudaMalloc on its per-step path (a device allocation may synchronise the
// device and stall every other stream).  For them the step can run out of a
// fixed scratch array that the library owns.  The array lives in device
// memory from the moment this library's device code is loaded on a GPU until
// the process exits, on every GPU that loads it.

namespace {

constexpr size_t kNoAllocScratchBytes = size_t(64) << 20;  // 64 MiB per device

static __device__ __align__(256) uint8_t g_step_scratch[kNoAllocScratchBytes];

std::mutex g_scratch_mu;
void* g_scratch_addr[kMaxDevices] = {};

// Device address of g_step_scratch on the current device, looked up once per
// device (host code must not pass the symbol itself to a kernel: on the host
// it names a stand-in, not device memory).
int scratch_address(void** out) {
  const int dev = current_device();
  if (dev < 0) return MS_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_scratch_mu);
  if (g_scratch_addr[dev] == nullptr) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_step_scratch) != cudaSuccess || p == nullptr) return MS_ERR_CUDA;
    g_scratch_addr[dev] = p;
  }
  *out = g_scratch_addr[dev];
  return MS_OK;
}

}  // namespace

extern "C" MS_API int ms_mixed_step_attention_noalloc(const void* q_rot, const void* k_cache, const void* v_cache,
                                                      int32_t num_pages, const int32_t* cu_seqlens_q,
                                                      const int32_t* q_start_pos, const int32_t* context_lens,
                                                      const int32_t* block_tables, int32_t bt_stride,
                                                      int32_t num_rows, int32_t num_tokens, int64_t context_total,
                                                      int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                                                      float scale, void* out, int32_t* dev_status,
                                                      ms_stream_t stream) {
  if (num_rows < 0 || num_tokens < 0 || context_total < 0 || H_q < 1 || H_kv < 1 || H_q % H_kv != 0 ||
      (D != 64 && D != 128))
    return MS_ERR_ARG;
  const size_t need = ws_layout(num_rows, num_tokens, context_total, H_q, H_kv, D).total;
  if (need > kNoAllocScratchBytes) return MS_ERR_SCRATCH;
  void* scratch = nullptr;
  const int rc0 = scratch_address(&scratch);
  if (rc0 != MS_OK) return rc0;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // The array keeps the previous call's contents.  The prologue zeroes its
  // status word before this call can set a bit (it also resets the queue
  // counters); no separate clearing launch sits between the append and the
  // prologue, so the prologue still overlaps the append.
  bool launched = false;
  const int rc = attention_call(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens,
                                block_tables, nullptr, 0, bt_stride, num_rows, num_tokens, context_total, H_q, H_kv, D,
                                page_size, scale, out, scratch, kNoAllocScratchBytes, stream, true, 0, &launched);
  if (rc != MS_OK) return rc;
  if (dev_status != nullptr) {
    const cudaError_t e = launched ? cudaMemcpyAsync(dev_status, scratch, sizeof(int32_t), cudaMemcpyDeviceToDevice, st)
                                   : cudaMemsetAsync(dev_status, 0, sizeof(int32_t), st);
    if (e != cudaSuccess) return MS_ERR_CUDA;
  }
  return MS_OK;
}
