// Mixed-batch attention over a paged 4-bit K/V cache (q4.cuh), sm_103a.
//
// The same step as attention.cu, with the same prologue, queues and split of
// the SMs.  What changes is where K and V come from:
//
//   chunk rows (d > 1): chunk_phase with four more warps, which read pages and
//     write their values into the shared-memory tiles.
//   decode rows (d = 1): 16 worker warps in teams, each warp with a private ring
//     of pages in shared memory filled by bulk copies, one a page.  A page of K
//     and V is 2.25 KB instead of 8 KB, so the time goes into instructions rather
//     than bytes, and the codes go into the tensor cores undecoded as far as the
//     algebra allows.  With x the codes of a group, n = x + 8 its nibbles and s
//     its scale,
//         q . K = sum_g s_g (q_g . x_g) = sum_g s_g (q_g . (128 + n_g) - 136 sum q_g):
//     the operand is the bf16 pair 128 + n, one shift and one logic instruction
//     for two values, and the offsets' share is one more product, of the scales as
//     they are stored with the sums.  For V the scales go into the weights,
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
// The cost model's rates (attention_step.cuh), measured at D = 128 and used for both
// head dims.  In a build that forced the split for the purpose, the one that they
// choose was within 1 % of the best of 13 on six mixed steps (124 to 2140 us).
constexpr float kQ4TileCycles = 4900.f;
constexpr float kQ4DecodeBytesPerCycle = 24.f;

// Decode phase's shared memory: every warp's ring of NST stages of two pages,
// what the teams know of their splits, the rings' barriers.
template <int D>
struct DecQ4 {
  static constexpr int WARPS = kQ4Threads / 32;
  static constexpr int NST = 3;
  static constexpr int PAGE = Q4<D>::BYTES;
  static constexpr int STAGE = 2 * PAGE;
  static constexpr int TEAM_OFF = WARPS * NST * STAGE;
  static constexpr int BAR_OFF = TEAM_OFF + WARPS / 2 * 64;  // a Team each
  static constexpr int SMEM = BAR_OFF + WARPS * NST * 8;
};

// One split (row, KV head, pages [p0, p0 + np) of the row), as its team's first
// warp looked it up; np == 0: the queue is empty.
struct __align__(16) Split {
  int row, k, hk, tok;   // k: the row's position among the decode rows
  int p0, np, keys, ns;  // keys: from page p0 to the row's end; ns: splits of the row
  int part;              // record of the split's first head
};
struct __align__(16) Team {
  Split split;
  int failed, last;  // a wait of the team gave up; the split is its row's last to finish
};

// D = A B, from zero
__device__ __forceinline__ void mma_16816_bf16_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Part i of a number as the sum of three bf16 (24 bits of it): the rounded
// number, the rounded remainder, and what is left.
__device__ __forceinline__ float bf16_part(float x, int i) {
  for (int j = 0; j < i; ++j) x -= __bfloat162float(__float2bfloat16_rn(x));
  return __bfloat162float(__float2bfloat16_rn(x));
}

// The issue side of a warp's ring.
struct IssueCursor {
  const uint8_t* base;  // the pool at the split's KV head
  const int32_t* btr;   // the warp's first page-table entry
  int left, next;       // pages not yet asked for, pages asked for
  int ids, ids_next;    // lane j: page ids of this window of 32 pages and of the next
};

// Decode phase: teams of warps (2, 4, 8 or 16 of the CTA, as the prologue chose)
// pull splits until the queue is empty.  Each warp of a team runs its share of
// the split's pages by itself, in pairs -- one wait and one vote for 32 keys --
// and the team joins the results in shared memory, where the rings were.  A warp
// to a split would need no joining but many more splits: with few or long rows
// its pages keep it for tens of microseconds while other warps idle, and one
// warp joins the row's records at the end.  256 rows of 8 KV heads and 700 to
// 16384 keys: 372 us with a warp to a split of 64 pages, 310 us with four to 512;
// 61 rows of 1 to 5003 keys, 2 KV heads, D = 64: 55 us, and 20 us with eight to 32.
//
// Instructions are nearest to a limit: about 355 a page and warp (2.25 KB of K and V
// at D = 128), half of them on the logic pipe, which is 65 % busy, as are the
// issue slots; DRAM delivers 4.8 TB/s, 0.70 of the measured copy rate (256 rows,
// above).  Neither is full: with four warps to a scheduler, dependent steps and
// the pipe's turns leave the rest.  64 rows of 32 heads of their own and 512 to 4096
// keys: 122 us, 4.2 TB/s, issue slots 60 % busy.  Measured and not kept: shifts as multiplications (310 -> 362 to 388 us);
// V's offset taken off by a product with -136 instead of before it (330 us);
// one page at a time; 16-byte asynchronous copies by all lanes instead of a bulk
// copy a page (346 us before the teams, 378 us).
template <int D, int G>
__device__ __forceinline__ void decode_phase_q4(const AttnParams& p, uint8_t* dsmem) {
  using Q = Q4<D>;
  using C = DecQ4<D>;
  constexpr int NG = Q::NG, NST = C::NST, NK = D / 16;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int gq = lane >> 2, tq = lane & 3;
  // Row of a page that MMA token gq stands for: tokens 2 and 3, and 6 and 7, trade places, so that
  // the four rows that one load of V touches lie on both halves of the 128-byte lines
  const int ra = gq ^ ((gq >> 1) & 1);
  const uint32_t ring = smem_u32(dsmem) + warp * NST * C::STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(dsmem + C::BAR_OFF) + warp * NST;
  if (lane == 0) {
    for (int i = 0; i < NST; ++i) mbar_init(full + i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  const int n_items = p.hdr[H_NDEC_ITEMS];
  IssueCursor iss{};
  // The next pair of the warp's pages (the last may be alone) into stage `st`,
  // one bulk copy a page from lanes 0 and 1.
  int in_flight = 0;
  auto issue_pair = [&](int st) {
    if (iss.left == 0) return;
    const int w = iss.next & 31, n = min(iss.left, 2);
    if (w == 0) {
      iss.ids = iss.ids_next;
      iss.ids_next = lane + 32 < iss.left ? __ldg(iss.btr + iss.next + 32 + lane) : 0;
    }
    int phys = __shfl_sync(0xffffffffu, iss.ids, w + lane);  // lanes 0 and 1: the pair's pages
    if (lane == 0) mbar_arrive_expect_tx(full + st, n * C::PAGE);
    __syncwarp();
    if (lane < n) {
      if (phys < 0 || phys >= p.num_pages) {
        atomicOr(p.hdr + H_STATUS, MS_STATUS_BAD_PAGE);
        phys = 0;
      }
      bulk_g2s(dsmem + (warp * NST + st) * C::STAGE + lane * C::PAGE,
               iss.base + static_cast<int64_t>(phys) * p.H_kv * Q::BYTES, C::PAGE, full + st);
    }
    iss.next += n;
    iss.left -= n;
    ++in_flight;
  };
  bool failed = false;
  int st = 0;       // stage of the next pair
  uint32_t ph = 0;  // its parity
  auto next_stage = [&]() {
    if (++st == NST) {
      st = 0;
      ph ^= 1u;
    }
  };
  // The warp's pages, np of them with `rem` keys from the first to the row's end.  Leaves O^T in acc -- the lane holds elements 32 g + 8 (gq / 2) + 2 i +
  // gq % 2 of heads 2 tq and 2 tq + 1, with i = 2 m in acc[2 g + m][0, 1] and
  // i = 2 m + 1 in acc[2 g + m][2, 3] -- and those heads' reference maxima (in
  // log2 units) and sums.
  float acc[NK][4], mu0, mu1, l0, l1;
  const float sl2 = p.scale_log2;
  constexpr float kRescaleLog2 = 8.f;  // raise the reference max only when it grows by 2^8
  auto run_pages = [&](int tok, int hk, int np, int rem) {
    // B operand of S^T = K Q^T: lane (head gq, quarter tq) holds the eight elements of quarter tq
    // of every group.  The offsets' share of the scores, sum_g s_g (-136 sum q_g), is a product
    // over the groups too: its B operand holds -136 sum q_g in three bf16 parts, column by column
    // the groups of part 0, of part 1, ..., against the row's scales as they are stored.
    uint32_t qb[NG][4], ob0, ob1 = 0u;
    {
      const bf16* q = p.q_rot + (static_cast<int64_t>(tok) * p.H_q + hk * G + gq) * D + 8 * tq;
      float off[NG];
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (gq < G) x = __ldg(reinterpret_cast<const uint4*>(q + 32 * g));
        qb[g][0] = x.x; qb[g][1] = x.y; qb[g][2] = x.z; qb[g][3] = x.w;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum += bf16_lo(qb[g][i]) + bf16_hi(qb[g][i]);
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        off[g] = -136.f * sum;
      }
      if constexpr (NG == 4) {
        const float x = tq & 1 ? off[2] : off[0], y = tq & 1 ? off[3] : off[1];
        const __nv_bfloat162 lo = __floats2bfloat162_rn(bf16_part(x, tq >> 1), bf16_part(y, tq >> 1));
        const __nv_bfloat162 hi = __floats2bfloat162_rn(bf16_part(x, 2), bf16_part(y, 2));
        ob0 = *reinterpret_cast<const uint32_t*>(&lo);
        if (tq < 2) ob1 = *reinterpret_cast<const uint32_t*>(&hi);
      } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(bf16_part(off[0], tq), bf16_part(off[1], tq));
        ob0 = tq < 3 ? *reinterpret_cast<const uint32_t*>(&lo) : 0u;
      }
    }
#pragma unroll
    for (int j = 0; j < NK; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
    mu0 = mu1 = -INFINITY;
    l0 = l1 = 0.f;
    for (int pi = 0; pi < np; pi += 2, rem -= 2 * kPage) {
      __syncwarp();  // every lane is done with the stage before
      issue_pair(st == 0 ? NST - 1 : st - 1);
      // a lane whose wait gave up goes on within the stage's bounds to the vote below
      const bool late = !mbar_wait(full + st, ph, nullptr);  // 2 s: a limit from the parameters costs registers
      const uint32_t stage = ring + st * C::STAGE;
      const int n_half = pi + 1 < np ? 2 : 1;
      // S^T: lane holds (row ra, heads 2 tq, 2 tq + 1) and (row ra + 8, same heads) of each page
      float s[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[h][0] = s[h][1] = s[h][2] = s[h][3] = 0.f;
        if (h < n_half) {
          const uint32_t pg = stage + h * C::PAGE;
          uint32_t ka[NG], kb[NG], sa[NG / 2], sb[NG / 2];
          lds_words<NG>(pg + ra * Q::ROW + tq * 4 * NG, ka);
          lds_words<NG>(pg + (ra + 8) * Q::ROW + tq * 4 * NG, kb);
          lds_words<NG / 2>(pg + Q::KS_OFF + ra * NG * 2, sa);
          lds_words<NG / 2>(pg + Q::KS_OFF + (ra + 8) * NG * 2, sb);
          const uint32_t s_a = NG == 4 && (tq & 1) ? sa[NG / 2 - 1] : sa[0], s_b = NG == 4 && (tq & 1) ? sb[NG / 2 - 1] : sb[0];
          const uint32_t sc[4] = {s_a, s_b, s_a, s_b};
          mma_16816_bf16_zero(s[h], sc, ob0, ob1);
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float c[4];
            const uint32_t a[4] = {q4_pair128(ka[g], 0), q4_pair128(kb[g], 0), q4_pair128(ka[g], 1), q4_pair128(kb[g], 1)};
            mma_16816_bf16_zero(c, a, qb[g][0], qb[g][1]);
            const uint32_t a2[4] = {q4_pair128(ka[g], 2), q4_pair128(kb[g], 2), q4_pair128(ka[g], 3), q4_pair128(kb[g], 3)};
            mma_16816_bf16(c, a2, qb[g][2], qb[g][3]);
            const float fa = g & 1 ? bf16_hi(sa[g >> 1]) : bf16_lo(sa[g >> 1]);
            const float fb = g & 1 ? bf16_hi(sb[g >> 1]) : bf16_lo(sb[g >> 1]);
            s[h][0] = fmaf(fa, c[0], s[h][0]);
            s[h][1] = fmaf(fa, c[1], s[h][1]);
            s[h][2] = fmaf(fb, c[2], s[h][2]);
            s[h][3] = fmaf(fb, c[3], s[h][3]);
          }
        }
      }
      if (n_half == 1) s[1][0] = s[1][1] = s[1][2] = s[1][3] = -INFINITY;
      if (rem < 2 * kPage) {  // the row's last keys
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h * kPage + ra >= rem) s[h][0] = s[h][1] = -INFINITY;
          if (h * kPage + ra + 8 >= rem) s[h][2] = s[h][3] = -INFINITY;
        }
      }
      // the lanes compare their own scores with the reference maximum; only when one of them is
      // past it by more than 2^8 do they look for the heads' maxima
      float mh0 = fmaxf(fmax3(s[0][0], s[0][2], s[1][0]), s[1][2]) * sl2;
      float mh1 = fmaxf(fmax3(s[0][1], s[0][3], s[1][1]), s[1][3]) * sl2;
      if (__any_sync(0xffffffffu, late || mh0 > mu0 + kRescaleLog2 || mh1 > mu1 + kRescaleLog2)) {
        if (__any_sync(0xffffffffu, late)) {
          failed = true;
          break;
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mh0 = fmaxf(mh0, __shfl_xor_sync(0xffffffffu, mh0, o));
          mh1 = fmaxf(mh1, __shfl_xor_sync(0xffffffffu, mh1, o));
        }
        const bool g0 = mh0 > mu0 + kRescaleLog2, g1 = mh1 > mu1 + kRescaleLog2;
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
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[h][0] = ex2(fmaf(s[h][0], sl2, -mu0));
        s[h][1] = ex2(fmaf(s[h][1], sl2, -mu1));
        s[h][2] = ex2(fmaf(s[h][2], sl2, -mu0));
        s[h][3] = ex2(fmaf(s[h][3], sl2, -mu1));
        l0 += s[h][0] + s[h][2];
        l1 += s[h][1] + s[h][3];
      }
      --in_flight;
      next_stage();
      // O^T += V^T (P s)^T, page by page and group by group.  The weights p s are rounded to bf16, the operands'
      // type (2^-9 of each, independent from key to key); the sum l is of the unrounded p.  They stay finite while
      // V's scales are below 2^119, as they are wherever keys * max |V| < 2^120 keeps the sums finite (p <= 2^8).
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h >= n_half) break;
        const uint32_t pg = stage + h * C::PAGE + Q::V_OFF;
        uint32_t v[4][NG / 2], wa[NG / 2], wb[NG / 2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // MMA tokens 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9
          const int r = 2 * tq + ((i & 1) ^ (tq & 1)) + 8 * (i >> 1);
          lds_words<NG / 2>(pg + r * Q::ROW + gq * 2 * NG, v[i]);
        }
        lds_words<NG / 2>(pg + Q::VS_OFF - Q::V_OFF + ra * NG * 2, wa);
        lds_words<NG / 2>(pg + Q::VS_OFF - Q::V_OFF + (ra + 8) * NG * 2, wb);
        if (rem < 2 * kPage) {  // rows past the context may hold any scale: their weight is 0
#pragma unroll
          for (int j = 0; j < NG / 2; ++j) {
            if (h * kPage + ra >= rem) wa[j] = 0u;
            if (h * kPage + ra + 8 >= rem) wb[j] = 0u;
          }
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float fa = g & 1 ? bf16_hi(wa[g >> 1]) : bf16_lo(wa[g >> 1]);
          const float fb = g & 1 ? bf16_hi(wb[g >> 1]) : bf16_lo(wb[g >> 1]);
          const float2 w01 = fmul2(make_float2(s[h][0], s[h][1]), make_float2(fa, fa));
          const float2 w23 = fmul2(make_float2(s[h][2], s[h][3]), make_float2(fb, fb));
          const __nv_bfloat162 h01 = __floats2bfloat162_rn(w01.x, w01.y), h23 = __floats2bfloat162_rn(w23.x, w23.y);
          const uint32_t b0 = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h01));
          const uint32_t b1 = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&h23));
          const uint32_t lo = join_halves(v[0][g >> 1], v[1][g >> 1], g & 1);
          const uint32_t hi = join_halves(v[2][g >> 1], v[3][g >> 1], g & 1);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const uint32_t a[4] = {q4_pair(lo, 2 * m), q4_pair(lo, 2 * m + 1), q4_pair(hi, 2 * m), q4_pair(hi, 2 * m + 1)};
            mma_16816_bf16(acc[2 * g + m], a, b0, b1);
          }
        }
      }
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
  };
  const int d0 = 8 * (gq >> 1) + (gq & 1);  // the lane's first element

  const int T = p.hdr[H_TEAM], team = warp / T, tw = warp - team * T, tt = threadIdx.x - team * T * 32;
  static_assert(sizeof(Team) <= 64, "team words");
  Team* tm = reinterpret_cast<Team*>(dsmem + C::TEAM_OFF) + team;
  const Split* split = &tm->split;
  float* s_acc = reinterpret_cast<float*>(dsmem + team * T * NST * C::STAGE);  // [warp][head][D]
  float* s_ml = s_acc + T * G * D;                                             // [warp][head][max, sum]
  static_assert(G * (D + 2) * 4 <= NST * C::STAGE, "a warp's joined results exceed its ring");
  auto team_sync = [&]() { named_bar_sync(1 + team, T * 32); };
  // The team's first warp looks the next split up: its id, its table entry, then
  // the row's words together, each step while the team is at something else.
  // The id is not taken before the team has run its pages: it would be held back
  // from a team that is free sooner.
  int id = 0;
  int2 entry = make_int2(0, 0);
  auto take_id = [&]() {
    if (tt == 0) id = atomicAdd(p.hdr + H_DEC_CTR, 1);
  };
  auto load_entry = [&]() {
    if (tw != 0) return;
    id = __shfl_sync(0xffffffffu, id, 0);
    if (id < n_items) entry = __ldg(p.dec_items + id / p.H_kv);  // (decode row and row, split)
  };
  auto load_split = [&]() {
    if (tw != 0) return;
    Split x{};
    if (id < n_items) {
      const int size = p.hdr[H_SPLIT];
      x.hk = id % p.H_kv;
      x.k = entry.x & 0xffff;
      x.row = entry.x >> 16;
      const int ctx = __ldg(p.ctx_lens + x.row);
      x.tok = __ldg(p.cu + x.row);
      x.ns = __ldg(p.dec_nsplit + x.k);
      x.part = __ldg(p.dec_part_base + x.k) + entry.y * p.H_q + x.hk * G;
      x.p0 = entry.y * size;
      x.np = min(size, (ctx + kPage - 1) / kPage - x.p0);
      x.keys = ctx - x.p0 * kPage;
    }
    if (lane == 0) tm->split = x;
  };
  if (tt == 0) tm->failed = 0;
  take_id();
  load_entry();
  load_split();
  team_sync();
  while (split->np > 0) {
    {
      const int np = split->np, hk = split->hk;
      const int share = 2 * ((np + 2 * T - 1) / (2 * T));  // pages to a warp, in pairs
      const int w0 = tw * share, mine = max(0, min(share, np - w0));
      iss.left = p.test_stall != 0 ? 0 : mine;  // test hook: no copy is issued, and the wait for it gives up
      iss.next = 0;
      iss.base = p.kv_q4 + hk * Q::BYTES;
      iss.btr = row_table(p, split->row) + split->p0 + w0;
      iss.ids_next = lane < mine ? __ldg(iss.btr + lane) : 0;
#pragma unroll 1
      for (int i = 0, s0 = st; i < NST - 1; ++i, s0 = s0 == NST - 1 ? 0 : s0 + 1) issue_pair(s0);
      run_pages(split->tok, hk, mine, split->keys - w0 * kPage);
    }
    take_id();
    const int tok = split->tok, hk = split->hk, k = split->k, ns = split->ns, part = split->part;
    if (failed && lane == 0) tm->failed = 1;
    team_sync();  // every warp is done with its ring, and with the split's words
    if (tm->failed) {
      failed = true;
      break;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int hh = 2 * tq + x;
      if (hh >= G) continue;
      float* dst = s_acc + (tw * G + hh) * D + d0;
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        dst[32 * (j >> 1) + 4 * (j & 1)] = acc[j][x];
        dst[32 * (j >> 1) + 4 * (j & 1) + 2] = acc[j][2 + x];
      }
      if (gq == 0) {
        s_ml[(tw * G + hh) * 2] = x == 0 ? mu0 : mu1;
        s_ml[(tw * G + hh) * 2 + 1] = x == 0 ? l0 : l1;
      }
    }
    team_sync();
    for (int c = tt; c < G * D; c += T * 32) {
      const int hh = c / D;
      float M = -INFINITY, L = 0.f, o = 0.f;
#pragma unroll 4
      for (int w = 0; w < T; ++w) M = fmaxf(M, s_ml[(w * G + hh) * 2]);
#pragma unroll 4
      for (int w = 0; w < T; ++w) {
        const float x = ex2(s_ml[(w * G + hh) * 2] - M);
        L += x * s_ml[(w * G + hh) * 2 + 1];
        o += x * s_acc[w * G * D + c];
      }
      if (ns == 1) {
        p.out[(static_cast<int64_t>(tok) * p.H_q + hk * G) * D + c] = __float2bfloat16_rn(o / L);
      } else {
        p.part_acc[static_cast<int64_t>(part) * D + c] = o;
        if (c % D == 0) *reinterpret_cast<float2*>(p.part_ml + (static_cast<int64_t>(part) + hh) * 2) = make_float2(M, L);
      }
    }
    fence_proxy_async_smem();  // the joined results are ordered before the next split's copies
    load_entry();
    if (ns > 1) {
      __threadfence();  // this split's records are visible before it is counted
      team_sync();
      if (tt == 0) tm->last = atomicAdd(p.dec_cnt + k * p.H_kv + hk, 1) == ns - 1;
      load_split();
      team_sync();
      if (tm->last) {
        __threadfence();
        for (int hh = tw; hh < G; hh += T) merge_splits<D, 16>(p, k, hk * G + hh, 1, tok, ns, lane);
      }
    } else {
      load_split();
      team_sync();
    }
  }
  if (failed) {
    if (lane == 0) atomicOr(p.hdr + H_STATUS, MS_STATUS_TIMEOUT);
    // let copies already in flight land before the CTA's shared memory is released
    for (; in_flight > 0; --in_flight) {
      mbar_wait(full + st, ph, nullptr, 200000000ull);
      next_stage();
    }
  }
  __syncwarp();
  if (lane == 0)
    for (int i = 0; i < NST; ++i) mbar_inval(full + i);
}

// One persistent CTA per SM, as attention_kernel.
template <int D, int G>
__global__ void __launch_bounds__(kQ4Threads, 1) attention_q4_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ AttnParams p) {
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
    if (!chunk && n_dec_items > 0) {
      decode_phase_q4<D, G>(p, smem);
      __syncthreads();
    } else if (chunk && n_ch_items > 0) {
      chunk_phase<D, G, kQ4>(&tm_q, &tm_q, &tm_q, &tm_q, p, smem, tmem);
      tc_fence_before();
      __syncthreads();
      ChBars* bars = reinterpret_cast<ChBars*>(smem + ChCfg<D>::BAR_OFF);
      const bool aborted = bars->abort != 0;
      if (threadIdx.x == 0) close_chunk_barriers(bars, &bars->raw_empty[kRawStages - 1]);
      __syncthreads();
      if (aborted) break;
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
  constexpr int smem = ChQ4<D>::SMEM > DecQ4<D>::SMEM ? ChQ4<D>::SMEM : DecQ4<D>::SMEM;
  static_assert(smem <= 232448, "attention kernel exceeds the per-CTA shared-memory limit");
  const int slot = (D == 128 ? 4 : 0) + (G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3);  // one bit per instance
  if (ensure_smem_limit(attention_q4_kernel<D, G>, slot, smem) != MS_OK) return MS_ERR_CUDA;
  if (launch_dependent(attention_q4_kernel<D, G>, dim3(p.num_sms), dim3(kQ4Threads), smem, st, tq, p) != cudaSuccess)
    return MS_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}

}  // namespace

extern "C" MS_API size_t ms_attention_workspace_size_q4(int32_t max_rows, int32_t max_tokens, int64_t max_context_total,
                                                        int32_t H_q, int32_t H_kv, int32_t D) {
  const size_t n = ms_attention_workspace_size(max_rows, max_tokens, max_context_total, H_q, H_kv, D);
  return n == 0 ? 0 : align_up(n, 256) + parts_total(max_tokens, H_q, H_kv, D);
}

namespace {

// The attention call over a 4-bit pool; stall_limit_ns as in step_setup (its decode phase issues no copy either).
int attention_q4_call(const void* q_rot, const void* kv_cache, int32_t num_pages, const int32_t* cu_seqlens_q,
                      const int32_t* q_start_pos, const int32_t* context_lens, const int32_t* block_tables,
                      const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride, int32_t num_rows, int32_t num_tokens,
                      int64_t context_total, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size, float scale, void* out,
                      void* workspace, size_t ws_bytes, int64_t stall_limit_ns, ms_stream_t stream) {
  AttnParams p;
  bool empty = true;
  int rc = step_setup(q_rot, kv_cache, kv_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables,
                      bt_offsets, bt_offsets != nullptr ? bt_len : 0, bt_offsets != nullptr ? 0 : bt_stride, num_rows,
                      num_tokens, context_total, H_q, H_kv, D, page_size, scale, out, workspace, ws_bytes, false,
                      stall_limit_ns, &p, &empty);
  if (rc != MS_OK || empty) return rc;
  p.kv_q4 = static_cast<const uint8_t*>(kv_cache);
  p.dec_workers = p.num_sms * (kQ4Threads / 32);
  p.tile_cycles = kQ4TileCycles;
  p.dec_bytes_cycle = kQ4DecodeBytesPerCycle;
  p.key_bytes = q4_block_bytes(D) / 16.f;
  set_parts_room(&p, workspace, ws_bytes, context_total);
  EncodeTiledFn enc = get_encode_fn();
  if (enc == nullptr) return MS_ERR_CUDA;
  CUtensorMap tq;
  const cuuint64_t dq[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H_q), static_cast<cuuint64_t>(num_tokens)};
  const cuuint64_t sq[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H_q) * D * 2};
  const cuuint32_t bq[3] = {64, static_cast<cuuint32_t>(p.G), static_cast<cuuint32_t>(128 / p.G)};
  if (!encode_bf16(enc, &tq, q_rot, 3, dq, sq, bq)) return MS_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = launch_prologue<true>(p, st);
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

}  // namespace

extern "C" MS_API int ms_mixed_step_attention_q4(const void* q_rot, const void* kv_cache, int32_t num_pages,
                                                 const int32_t* cu_seqlens_q, const int32_t* q_start_pos,
                                                 const int32_t* context_lens, const int32_t* block_tables,
                                                 const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride,
                                                 int32_t num_rows, int32_t num_tokens, int64_t context_total, int32_t H_q,
                                                 int32_t H_kv, int32_t D, int32_t page_size, float scale, void* out,
                                                 void* workspace, size_t ws_bytes, ms_stream_t stream) {
  return attention_q4_call(q_rot, kv_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables, bt_offsets,
                           bt_len, bt_stride, num_rows, num_tokens, context_total, H_q, H_kv, D, page_size, scale, out,
                           workspace, ws_bytes, 0, stream);
}

extern "C" MS_API int ms_test_attention_stall_q4(const void* q_rot, const void* kv_cache, int32_t num_pages,
                                                 const int32_t* cu_seqlens_q, const int32_t* q_start_pos,
                                                 const int32_t* context_lens, const int32_t* block_tables,
                                                 int32_t bt_stride, int32_t num_rows, int32_t num_tokens,
                                                 int64_t context_total, int32_t H_q, int32_t H_kv, int32_t D,
                                                 int32_t page_size, float scale, void* out, void* workspace,
                                                 size_t ws_bytes, int64_t wait_limit_ns, ms_stream_t stream) {
  if (wait_limit_ns < 100000 || wait_limit_ns > 2000000000ll) return MS_ERR_ARG;  // 0.1 ms .. 2 s
  return attention_q4_call(q_rot, kv_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables, nullptr, 0,
                           bt_stride, num_rows, num_tokens, context_total, H_q, H_kv, D, page_size, scale, out, workspace,
                           ws_bytes, wait_limit_ns, stream);
}
