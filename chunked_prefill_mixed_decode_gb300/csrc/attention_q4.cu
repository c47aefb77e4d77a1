// Mixed-batch attention over a paged 4-bit K/V cache (q4.cuh), sm_103a.
//
// The same step as attention.cu, with the same prologue, queues and split of
// the SMs.  What changes is where K and V come from:
//
//   chunk rows (d > 1): chunk_phase with four more warps, which read pages and
//     write their values into the shared-memory tiles.
//   decode rows (d = 1): 16 worker warps, each with a private ring of pages in
//     shared memory filled by 16-byte asynchronous copies.  A page of K and V is
//     2.25 KB instead of 8 KB, so the time goes into instructions rather than
//     bytes, and the codes go into the tensor cores undecoded as far as the
//     algebra allows.  With x the codes of a group, n = x + 8 its nibbles and s
//     its scale,
//         q . K = sum_g s_g (q_g . x_g) = sum_g s_g (q_g . (128 + n_g) - 136 sum q_g):
//     the operand is the bf16 pair 128 + n, one shift and one logic instruction
//     for two values, and -136 sum q_g, fixed for an item, is the accumulator's
//     start.  For V the scales go into the weights,
//         O_d = sum_j (p_j s_jg) x_jd,
//     and the codes are centred first (one subtraction for two values): an
//     accumulator that carried 128 per weight through a long row would lose the
//     small differences that remain.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "attention_step.cuh"
#include "chunk_phase.cuh"
#include "mixed_step.h"
#include "ptx.cuh"
#include "q4.cuh"

namespace {

constexpr int kQ4Threads = 32 * (kDequantWarp0 + kDequantWarps);
constexpr float kQ4TileCycles = 5820.f;
constexpr float kQ4DecodeBytesPerCycle = 24.f;

template <int D>
struct DecQ4 {
  static constexpr int WARPS = kQ4Threads / 32;
  static constexpr int NST = 4;  // ring stages per warp
  static constexpr int STAGE = Q4<D>::BYTES;
  static constexpr int SMEM = WARPS * NST * STAGE;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t src, uint32_t* dst) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(dst[0]), "=r"(dst[1]), "=r"(dst[2]), "=r"(dst[3]) : "r"(src) : "memory");
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(dst[0]), "=r"(dst[1]) : "r"(src) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(dst[0]) : "r"(src) : "memory");
}

// D = A B + C with C = (c0, c1) in both row halves
__device__ __forceinline__ void mma_16816_bf16_from(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                                    float c1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%10,%11};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1));
}

// Where the pages of the work items come from: the issue side of a warp's ring.
struct IssueCursor {
  const int32_t* btr;  // the item's first page-table entry
  int hk, np, next;    // KV head, pages, next page to issue
  int ids, ids_next;   // lane j: page ids of this window of 32 pages and of the next
};

// What the consumer needs of an item, broadcast by shuffles from the lane that
// holds it: lane i of every warp keeps the record of item slot i.
struct ItemRec {
  int tok, hk, k, part, ns, np, rem;  // rem: keys from the item's first page to the row's end
};

template <int D, int G>
__device__ __noinline__ void decode_phase_q4(const AttnParams& p, uint8_t* dsmem) {
  using Q = Q4<D>;
  using C = DecQ4<D>;
  constexpr int NG = Q::NG, NST = C::NST, NK = D / 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  const uint32_t ring = smem_u32(dsmem) + warp * NST * C::STAGE;
  const int n_items = p.hdr[H_NDEC_ITEMS];
  const int split = p.hdr[H_SPLIT];
  const int64_t page_bytes = static_cast<int64_t>(p.H_kv) * Q::BYTES;

  // the id of the item after the one being issued is fetched one item ahead
  auto dequeue = [&]() -> int {
    int v = 0;
    if (lane == 0) v = atomicAdd(p.hdr + H_DEC_CTR, 1);
    return __shfl_sync(0xffffffffu, v, 0);
  };
  ItemRec rec{};          // this lane's item record
  IssueCursor iss{};
  int n_issued = 0;       // items whose issue has begun
  int next_id = dequeue();
  bool more = next_id < n_items;
  auto begin_item = [&]() {
    const int e = next_id / p.H_kv;
    const int2 kl = __ldg(p.dec_items + e);  // (decode row index, split within the row)
    const int row = __ldg(p.dec_rows + kl.x);
    const int ctx = __ldg(p.ctx_lens + row);
    iss.hk = next_id - e * p.H_kv;
    const int p0 = kl.y * split;
    iss.np = min(split, (ctx + kPage - 1) / kPage - p0);
    iss.next = 0;
    iss.btr = row_table(p, row) + p0;
    iss.ids = lane < iss.np ? __ldg(iss.btr + lane) : 0;
    if (lane == (n_issued & (NST - 1))) {
      rec.tok = __ldg(p.cu + row);
      rec.hk = iss.hk;
      rec.k = kl.x;
      rec.part = __ldg(p.dec_part_base + kl.x) + kl.y * p.H_q + iss.hk * G;
      rec.ns = __ldg(p.dec_nsplit + kl.x);
      rec.np = iss.np;
      rec.rem = ctx - p0 * kPage;
    }
    ++n_issued;
    next_id = dequeue();
    more = next_id < n_items;
  };
  // One page into stage `st`; a committed group even where nothing is left, so
  // that the count of groups in flight stays fixed.  V's 16-byte chunks are
  // swizzled within their 128-byte lines: the four rows that one load of the PV
  // operand touches are two lines apart or on the same half of a line.
  auto issue = [&](int st) {
    if (iss.next >= iss.np && more) begin_item();
    if (iss.next < iss.np) {
      const int w = iss.next & 31;
      if (w == 0) {
        if (iss.next > 0) iss.ids = iss.ids_next;
        const int j = iss.next + 32 + lane;
        iss.ids_next = j < iss.np ? __ldg(iss.btr + j) : 0;
      }
      int phys = __shfl_sync(0xffffffffu, iss.ids, w);
      if (phys < 0 || phys >= p.num_pages) {
        if (lane == 0) atomicOr(p.hdr + H_STATUS, MS_STATUS_BAD_PAGE);
        phys = 0;
      }
      const uint8_t* src = p.kv_q4 + phys * page_bytes + iss.hk * Q::BYTES + lane * 16;
      const uint32_t dst = ring + st * C::STAGE;
      constexpr int NC = Q::V_OFF / 512;  // chunks of K (and of V) per lane
      const int sw = lane ^ (D == 128 ? (lane >> 2) & 6 : (lane >> 2) & 2);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        cp_async16(dst + lane * 16 + i * 512, src + i * 512);
        cp_async16(dst + Q::V_OFF + sw * 16 + i * 512, src + Q::V_OFF + i * 512);
      }
      if (lane < (Q::BYTES - Q::KS_OFF) / 16) cp_async16(dst + Q::KS_OFF + lane * 16, src + Q::KS_OFF);
      ++iss.next;
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < NST - 1; ++i) issue(i);

  int st = 0;      // stage of the next page
  for (int item = 0; item < n_issued; ++item) {
    const int slot = item & (NST - 1);
    const int np = __shfl_sync(0xffffffffu, rec.np, slot);
    int rem = __shfl_sync(0xffffffffu, rec.rem, slot);
    const int tok = __shfl_sync(0xffffffffu, rec.tok, slot), hk = __shfl_sync(0xffffffffu, rec.hk, slot);
    // B operand of S^T = K Q^T: lane (head gq, quarter tq) holds the eight elements of quarter tq
    // of every group; and the accumulators' starts for heads 2 tq, 2 tq + 1
    uint32_t qb[NG][4];
    float cs[NG][2];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (gq < G)
        x = __ldg(reinterpret_cast<const uint4*>(p.q_rot + (static_cast<int64_t>(tok) * p.H_q + hk * G + gq) * D + 32 * g + 8 * tq));
      qb[g][0] = x.x; qb[g][1] = x.y; qb[g][2] = x.z; qb[g][3] = x.w;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += bf16_lo(qb[g][i]) + bf16_hi(qb[g][i]);
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      cs[g][0] = -136.f * __shfl_sync(0xffffffffu, sum, 8 * tq);
      cs[g][1] = -136.f * __shfl_sync(0xffffffffu, sum, 8 * tq + 4);
    }
    float acc[NK][4];
#pragma unroll
    for (int j = 0; j < NK; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    float mu0 = -INFINITY, mu1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // heads 2 tq and 2 tq + 1
    constexpr float kRescaleLog2 = 8.f;  // raise the reference max only when it grows by 2^8
    for (int pi = 0; pi < np; ++pi, rem -= kPage) {
      cp_async_wait<NST - 2>();
      __syncwarp();  // every lane's copies are in, and every lane is done with the stage before
      issue((st + NST - 1) & (NST - 1));
      const uint32_t stage = ring + st * C::STAGE;
      st = (st + 1) & (NST - 1);
      // S^T: lane holds (token gq, heads 2 tq, 2 tq + 1) and (token gq + 8, same heads)
      uint32_t ka[NG], kb[NG], sa[NG / 2], sb[NG / 2];
      lds_words<NG>(stage + gq * Q::ROW + tq * 4 * NG, ka);
      lds_words<NG>(stage + (gq + 8) * Q::ROW + tq * 4 * NG, kb);
      lds_words<NG / 2>(stage + Q::KS_OFF + gq * NG * 2, sa);
      lds_words<NG / 2>(stage + Q::KS_OFF + (gq + 8) * NG * 2, sb);
      float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float c[4];
        uint32_t a[4] = {q4_pair128(ka[g], 0), q4_pair128(kb[g], 0), q4_pair128(ka[g], 1), q4_pair128(kb[g], 1)};
        mma_16816_bf16_from(c, a, qb[g][0], qb[g][1], cs[g][0], cs[g][1]);
        uint32_t a2[4] = {q4_pair128(ka[g], 2), q4_pair128(kb[g], 2), q4_pair128(ka[g], 3), q4_pair128(kb[g], 3)};
        mma_16816_bf16(c, a2, qb[g][2], qb[g][3]);
        const float fa = g & 1 ? bf16_hi(sa[g >> 1]) : bf16_lo(sa[g >> 1]);
        const float fb = g & 1 ? bf16_hi(sb[g >> 1]) : bf16_lo(sb[g >> 1]);
        s0 = fmaf(fa, c[0], s0);
        s1 = fmaf(fa, c[1], s1);
        s2 = fmaf(fb, c[2], s2);
        s3 = fmaf(fb, c[3], s3);
      }
      const float sl2 = p.scale_log2;
      const bool va = gq < rem, vb = gq + 8 < rem;
      s0 = va ? s0 * sl2 : -INFINITY;
      s1 = va ? s1 * sl2 : -INFINITY;
      s2 = vb ? s2 * sl2 : -INFINITY;
      s3 = vb ? s3 * sl2 : -INFINITY;
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
      // O^T += V^T (P s)^T, group by group.  Rows past the context may hold any scale: their weight is 0.
      uint32_t v[4][NG / 2], wa[NG / 2], wb[NG / 2];
      {
        const int swz = D == 128 ? 2 * tq : 2 * (tq >> 1);
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // tokens 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
          const int r = 2 * tq + (i & 1) + 8 * (i >> 1);
          const int byte = r * Q::ROW + gq * 2 * NG;
          lds_words<NG / 2>(stage + Q::V_OFF + (byte ^ (swz << 4)), v[i]);
        }
        lds_words<NG / 2>(stage + Q::VS_OFF + gq * NG * 2, wa);
        lds_words<NG / 2>(stage + Q::VS_OFF + (gq + 8) * NG * 2, wb);
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const float fa = va ? (g & 1 ? bf16_hi(wa[g >> 1]) : bf16_lo(wa[g >> 1])) : 0.f;
        const float fb = vb ? (g & 1 ? bf16_hi(wb[g >> 1]) : bf16_lo(wb[g >> 1])) : 0.f;
        const __nv_bfloat162 h01 = __floats2bfloat162_rn(p0 * fa, p1 * fa), h23 = __floats2bfloat162_rn(p2 * fb, p3 * fb);
        const uint32_t b0 = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h01));
        const uint32_t b1 = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h23));
        const uint32_t lo = join_halves(v[0][g >> 1], v[1][g >> 1], g & 1), hi = join_halves(v[2][g >> 1], v[3][g >> 1], g & 1);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          uint32_t a[4] = {q4_pair(lo, 2 * m), q4_pair(lo, 2 * m + 1), q4_pair(hi, 2 * m), q4_pair(hi, 2 * m + 1)};
          mma_16816_bf16(acc[2 * g + m], a, b0, b1);
        }
      }
    }
    // O^T: lane holds elements 32 g + 8 (gq / 2) + 2 i + gq % 2 of heads 2 tq, 2 tq + 1, with i = 2 m in
    // acc[2 g + m][0, 1] and i = 2 m + 1 in acc[2 g + m][2, 3]
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    const int part = __shfl_sync(0xffffffffu, rec.part, slot), ns = __shfl_sync(0xffffffffu, rec.ns, slot);
    const int k = __shfl_sync(0xffffffffu, rec.k, slot);
    const int d0 = 8 * (gq >> 1) + (gq & 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hh = 2 * tq + e;
      if (hh >= G) continue;
      const float L = e == 0 ? l0 : l1, M = e == 0 ? mu0 : mu1;
      if (ns == 1) {
        const float inv = 1.f / L;
        bf16* dst = p.out + (static_cast<int64_t>(tok) * p.H_q + hk * G + hh) * D + d0;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          dst[32 * (j >> 1) + 4 * (j & 1)] = __float2bfloat16_rn(acc[j][e] * inv);
          dst[32 * (j >> 1) + 4 * (j & 1) + 2] = __float2bfloat16_rn(acc[j][2 + e] * inv);
        }
      } else {
        const int64_t r = part + hh;
        float* dst = p.part_acc + r * D + d0;
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          dst[32 * (j >> 1) + 4 * (j & 1)] = acc[j][e];
          dst[32 * (j >> 1) + 4 * (j & 1) + 2] = acc[j][2 + e];
        }
        if (gq == 0) *reinterpret_cast<float2*>(p.part_ml + r * 2) = make_float2(M, L);
      }
    }
    if (ns > 1) {
      __threadfence();  // this split's records are visible before it is counted
      __syncwarp();
      int last = 0;
      if (lane == 0) last = atomicAdd(p.dec_cnt + k * p.H_kv + hk, 1) == ns - 1;
      last = __shfl_sync(0xffffffffu, last, 0);
      if (last) {
        __threadfence();
        merge_splits<D>(p, k, hk * G, G, tok, ns, lane);
      }
    }
  }
  cp_async_wait<0>();
}

// One persistent CTA per SM, as attention_kernel.
template <int D, int G>
__global__ void __launch_bounds__(kQ4Threads, 1) attention_q4_kernel(const __grid_constant__ CUtensorMap tm_q, AttnParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5;
  if ((smem_u32(smem) & 1023u) != 0) {
    griddep_wait();
    if (threadIdx.x == 0) atomicOr(p.hdr + H_STATUS, MS_STATUS_INTERNAL);
    return;
  }
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
  const long long clk0 = clock64();
  const uint64_t ns0 = globaltimer_ns();
  const int n_ch_items = p.hdr[H_NCH_ITEMS];
  const int n_dec_items = p.hdr[H_NDEC_ITEMS];
  __syncthreads();  // every thread holds the address before the phases reuse the memory
  uint32_t smid;
  asm volatile("mov.u32 %0, %%smid;" : "=r"(smid));
  const bool chunk_first = static_cast<int>(smid) < p.hdr[H_CHUNK_CTAS];
  for (int ph = 0; ph < 2; ++ph) {
    const bool chunk = (ph == 0) == chunk_first;
    if (chunk && n_ch_items > 0) {
      chunk_phase<D, G, true>(&tm_q, &tm_q, &tm_q, &tm_q, p, smem, tmem);
      tc_fence_before();
      __syncthreads();
      ChBars* bars = reinterpret_cast<ChBars*>(smem + ChCfg<D>::BAR_OFF);
      const bool aborted = bars->abort != 0;
      if (threadIdx.x == 0)
        for (uint64_t* b = &bars->q_full; b <= &bars->mma_done[2]; ++b) mbar_inval(b);
      __syncthreads();
      if (aborted) break;
    } else if (!chunk && n_dec_items > 0) {
      decode_phase_q4<D, G>(p, smem);
      fence_proxy_async_smem();  // the ring's copies are ordered before a chunk phase's TMA into the same memory
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

template <int D, int G>
int launch_q4(const AttnParams& p, const CUtensorMap& tq, cudaStream_t st) {
  constexpr int smem = ChCfg<D>::SMEM > DecQ4<D>::SMEM ? ChCfg<D>::SMEM : DecQ4<D>::SMEM;
  static_assert(smem <= 232448, "attention kernel exceeds the per-CTA shared-memory limit");
  const int slot = (D == 128 ? 4 : 0) + (G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3);  // one bit per instance
  if (ensure_smem_limit(attention_q4_kernel<D, G>, slot, smem) != MS_OK) return MS_ERR_CUDA;
  if (launch_dependent(attention_q4_kernel<D, G>, dim3(p.num_sms), dim3(kQ4Threads), smem, st, tq, p) != cudaSuccess)
    return MS_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}

}  // namespace

extern "C" MS_API int ms_mixed_step_attention_q4(const void* q_rot, const void* kv_cache, int32_t num_pages,
                                                 const int32_t* cu_seqlens_q, const int32_t* q_start_pos,
                                                 const int32_t* context_lens, const int32_t* block_tables,
                                                 const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride,
                                                 int32_t num_rows, int32_t num_tokens, int64_t context_total, int32_t H_q,
                                                 int32_t H_kv, int32_t D, int32_t page_size, float scale, void* out,
                                                 void* workspace, size_t ws_bytes, ms_stream_t stream) {
  AttnParams p;
  bool empty = true;
  int rc = step_setup(q_rot, kv_cache, kv_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables,
                      bt_offsets, bt_offsets != nullptr ? bt_len : 0, bt_offsets != nullptr ? 0 : bt_stride, num_rows,
                      num_tokens, context_total, H_q, H_kv, D, page_size, scale, out, workspace, ws_bytes, false, 0, &p,
                      &empty);
  if (rc != MS_OK || empty) return rc;
  p.kv_q4 = static_cast<const uint8_t*>(kv_cache);
  p.dec_workers = p.num_sms * (kQ4Threads / 32);
  p.tile_cycles = kQ4TileCycles;
  p.dec_bytes_cycle = kQ4DecodeBytesPerCycle;
  p.key_bytes = q4_block_bytes(D) / 16.f;
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return MS_ERR_CUDA;
  CUtensorMap tq;
  const cuuint64_t dq[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H_q), static_cast<cuuint64_t>(num_tokens)};
  const cuuint64_t sq[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H_q) * D * 2};
  const cuuint32_t bq[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(128 / p.G)};
  if (!encode_bf16(enc, &tq, q_rot, 3, dq, sq, bq)) return MS_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = launch_prologue(p, st);
  if (rc != MS_OK) return rc;
  switch (D * 100 + p.G) {
    case 6401: return launch_q4<64, 1>(p, tq, st);
    case 6402: return launch_q4<64, 2>(p, tq, st);
    case 6404: return launch_q4<64, 4>(p, tq, st);
    case 6408: return launch_q4<64, 8>(p, tq, st);
    case 12801: return launch_q4<128, 1>(p, tq, st);
    case 12802: return launch_q4<128, 2>(p, tq, st);
    case 12804: return launch_q4<128, 4>(p, tq, st);
    default: return launch_q4<128, 8>(p, tq, st);
  }
}
