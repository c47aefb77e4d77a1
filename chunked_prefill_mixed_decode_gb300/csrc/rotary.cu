// Rotary embedding in its other forms: frequencies scaled for long contexts (host),
// the table of a run of positions on the GPU, and the paged append with the rotation
// over part of a head, in halves or in neighbouring pairs.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "append_rope.cuh"
#include "device_state.cuh"
#include "mixed_step.h"
#include "ptx.cuh"

namespace {

using ms::fadd2;
using ms::ffma2;
using ms::fmul2;

constexpr int kMaxPairs = 64;  // rotary_dim / 2 at most

// ----------------------------------------------------------------------------
// frequencies (host)
// ----------------------------------------------------------------------------

constexpr double kTwoPi = 6.283185307179586476925286766559;

// The pair (a real number) that turns `turns` times over n positions: n base^(-2x/R) = 2 pi turns.
double pair_of_turns(double turns, double n, double base, double R) {
  return R * std::log(n / (turns * kTwoPi)) / (2.0 * std::log(base));
}

// f / (2 pi) modulo 1 in units of 2^-64, from 128 bits of 1 / (2 pi), to half a unit: row * unit,
// which wraps as turns do, is then the angle of any int32 position to 2^-34 turns and that of the first
// million to 2^-45.
uint64_t turns_fixed(double f) {
  constexpr uint64_t kHi = 0x28be60db9391054aull, kLo = 0x7f09d5f47d4d3770ull;  // 1 / (2 pi) times 2^128
  if (f == 0.0) return 0;
  int e = 0;
  const double m = std::frexp(std::fabs(f), &e);  // f = m 2^e, m in [1/2, 1)
  const uint64_t mant = static_cast<uint64_t>(std::ldexp(m, 53));
  const unsigned __int128 lo = static_cast<unsigned __int128>(mant) * kLo;
  const unsigned __int128 mid = static_cast<unsigned __int128>(mant) * kHi + static_cast<uint64_t>(lo >> 64);
  const int shift = 53 - e;  // f / (2 pi) 2^64 = mid 2^(e - 53)
  if (shift > 126) return 0;
  const unsigned __int128 r = shift > 0 ? ((mid >> (shift - 1)) + 1) >> 1 : mid << -shift;
  const uint64_t t = static_cast<uint64_t>(r);
  return f < 0 ? 0 - t : t;
}

// ----------------------------------------------------------------------------
// table (device)
// ----------------------------------------------------------------------------
//
// The angle of (position p, pair i) is p * turns[i] modulo 1 in 64-bit whole numbers, off by p times the
// frequency's last bit, (p + 1) 2^-65 turns at most.  It is split into the nearest quarter turn and a rest x
// of at most pi / 4, in two floats: of the rest's 62 bits the upper 45 are taken (2 pi 2^-47 left out), and the
// small part's own roundings are below that too, so that x is off by 2 pi 2^-46 at most beside the angle's error.
// Cosine and sine of x by their Taylor series in fp32 (the first term left out is below 3e-9), with the leading
// terms kept in two floats.  What the last rounding does not cause is the rounding of the cubic term's factors:
// 3.5 of them, 2^-24 each, of at most 0.115 of a sine.  A result is off by at most 0.8 * 2^-23 of its size (0.5 +
// 0.2 + 0.03) and by x's and the angle's error times the amplitude, which shows where a sine is below 1e-6: there
// it is several of its steps, if 1e-13 in all.  A rotation passes absolute errors on, so the 17 bits below are not
// carried in a third float.  (FP64 has 1/64 of the fp32 rate on this GPU.)

// The amplitude m in two floats, and m times the Taylor coefficients.
struct Series {
  float hi, lo, s3, s5, s7, s9, c2, c4, c6, c8, c10;
};

struct TableArgs {
  uint64_t turns[kMaxPairs];
  float* cos_tab;
  float* sin_tab;
  int64_t first;  // position of row 0
  int32_t n, half;
  Series m;
};

// Two pairs at a time, in the halves of float2s: a packed operation of two products or sums is one instruction,
// and instructions are what the kernel spends beside its 8 bytes a pair (131072 rows of 64 pairs, whose 67 MB stay in L2:
// 19.1 us one pair at a time, 13.4 now; with an amplitude 23.1, and 16.7 where cosines and sines were
// multiplied at the end, 14.6 with it in the series).
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg2(float2 x) { return make_float2(-x.x, -x.y); }

// The whole-number part of an angle, t of 2^64 turns: u holds the nearest quarter turn in its two top bits, and the
// rest (less an eighth of a turn) below them; upper and lower are the rest's upper 22 bits, signed, and next 23.
struct Rest {
  uint32_t u;
  float upper, lower;
};

__device__ __forceinline__ Rest split_turns(uint64_t t) {
  Rest r;
  r.u = static_cast<uint32_t>(t >> 32) + 0x20000000u;  // an eighth of a turn on: 4 quarters wrap to 0
  // whole numbers below 2^23 become floats as the mantissa of one whose step is 1
  r.upper = __uint_as_float(((r.u >> 8) & 0x3fffffu) | 0x4b000000u) - (8388608.f + 2097152.f);
  r.lower = __uint_as_float((__funnelshift_r(static_cast<uint32_t>(t), r.u, 17) & 0x7fffffu) | 0x4b000000u) - 8388608.f;
  return r;
}

// Cosine and sine of two angles, rounded, times an amplitude m.hi + m.lo (1 + 0 where not Scaled): m times the series,
// with m in its coefficients and the leading terms' products in two floats too.
template <bool Scaled>
__device__ __forceinline__ void cos_sin(uint64_t t0, uint64_t t1, const Series& m, float2& c_out, float2& s_out) {
  const Rest r0 = split_turns(t0), r1 = split_turns(t1);
  // x = 2 pi rest, |x| <= pi / 4, as the two floats x and y
  constexpr float kHi = 6.28318548202514648f, kLo = -1.74845553146951715e-7f;  // 2 pi
  const float2 a = make_float2(r0.upper, r1.upper), b = make_float2(r0.lower, r1.lower);
  const float2 p = fmul2(a, splat(kHi * 0x1p-24f));
  const float2 q = ffma2(b, splat(kHi * 0x1p-47f), ffma2(a, splat(kLo * 0x1p-24f), ffma2(a, splat(kHi * 0x1p-24f), neg2(p))));
  // their sum rounded, and what the rounding left out (|p| >= |q|, or p = 0)
  const float2 x = fadd2(p, q), y = fadd2(q, neg2(fadd2(x, neg2(p))));
  const float2 z = fmul2(x, x);
  const float2 z_lo = ffma2(fadd2(x, x), y, ffma2(x, x, neg2(z)));  // x^2 and what its rounding left out
  // sin x = x - x^3 / 3! + ...
  float2 ps = ffma2(z, splat(m.s9), splat(m.s7));
  ps = ffma2(z, ps, splat(m.s5));
  ps = ffma2(z, ps, splat(m.s3));
  float2 s_hi = x, s_left = y;
  if constexpr (Scaled) {
    s_hi = fmul2(x, splat(m.hi));
    s_left = ffma2(y, splat(m.hi), ffma2(x, splat(m.lo), ffma2(x, splat(m.hi), neg2(s_hi))));
  }
  const float2 s = fadd2(s_hi, ffma2(fmul2(z, x), ps, s_left));
  // cos x = 1 - x^2 / 2 + x^4 / 4! - ...
  float2 pc = ffma2(z, splat(m.c10), splat(m.c8));
  pc = ffma2(z, pc, splat(m.c6));
  pc = ffma2(z, pc, splat(m.c4));
  const float2 c_hi = ffma2(z, splat(m.c2), splat(m.hi));
  float2 c_left = ffma2(z_lo, splat(m.c2), ffma2(z, splat(m.c2), fadd2(splat(m.hi), neg2(c_hi))));
  if constexpr (Scaled) c_left = fadd2(c_left, ffma2(z, splat(-0.5f * m.lo), splat(m.lo)));
  const float2 c = fadd2(c_hi, ffma2(fmul2(z, z), pc, c_left));
  // by quarters: (c, s), (-s, c), (-c, -s), (s, -c)
  const auto turn = [](uint32_t u, float cc, float ss, float& co, float& so) {
    const bool odd = (u & 0x40000000u) != 0;
    const float x = odd ? ss : cc, y = odd ? cc : ss;
    co = __uint_as_float(__float_as_uint(x) ^ ((u + 0x40000000u) & 0x80000000u));
    so = __uint_as_float(__float_as_uint(y) ^ (u & 0x80000000u));
  };
  turn(r0.u, c.x, s.x, c_out.x, s_out.x);
  turn(r1.u, c.y, s.y, c_out.y, s_out.y);
}

// A thread makes four neighbouring pairs of every row `rows` apart and stores 16 bytes of each table.
template <bool Scaled>
__global__ void __launch_bounds__(256) rotary_table_kernel(const __grid_constant__ TableArgs a) {
  __shared__ uint64_t turns[kMaxPairs];  // lanes read different ones: from the parameters one after another
  if (threadIdx.x < kMaxPairs) turns[threadIdx.x] = a.turns[threadIdx.x];
  __syncthreads();
  const int quads = a.half >> 2, per_block = 256 / quads;  // rows of the block at a time
  const int r = threadIdx.x / quads, i0 = (threadIdx.x - r * quads) * 4;
  if (r >= per_block) return;
  const int64_t rows = static_cast<int64_t>(gridDim.x) * per_block;
  int64_t row = static_cast<int64_t>(blockIdx.x) * per_block + r;
  uint64_t t[4], step[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint64_t f = turns[i0 + j];
    t[j] = static_cast<uint64_t>(a.first + row) * f;
    step[j] = static_cast<uint64_t>(rows) * f;
  }
  for (; row < a.n; row += rows) {
    float2 c[2], s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) cos_sin<Scaled>(t[2 * j], t[2 * j + 1], a.m, c[j], s[j]);
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] += step[j];
    const int64_t at = row * a.half + i0;
    *reinterpret_cast<float4*>(a.cos_tab + at) = make_float4(c[0].x, c[0].y, c[1].x, c[1].y);
    *reinterpret_cast<float4*>(a.sin_tab + at) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
  }
}

// ----------------------------------------------------------------------------
// append (device)
// ----------------------------------------------------------------------------
//
// A warp takes heads of one token, 4 at a time (8 at D = 64): a lane owns the same two 16-byte
// chunks of every head and keeps the token's cosines and sines for them.  In halves a lane's
// chunks are a pair's two sides, R / 2 apart, or, past the rotary part, two chunks that are
// copied; in neighbouring pairs a chunk holds four whole pairs.  It has to move
// (4 H_q + 8 H_kv) D bytes a token and 4 R of the tables: 203 MB for 8192 tokens of 32 / 8 heads,
// D = 128, R = 64, in 34.8 us, 0.86 of the measured copy rate; 6000 tokens of 8 KV heads alone 10.2
// us, 0.71 (a replayed graph, inputs past L2).  What counts is bytes in flight: 64 to 80 KB an SM, by
// two groups of heads ahead in small blocks (four ahead, in blocks of 256: 41 us; one: 37.7; loads
// marked as streaming: 35.6; several warps a token, whose tables then count again: 50).

struct RotaryArgs {
  AppendArgs a;
  int64_t q_stride, k_stride, v_stride;  // elements from one token's rows to the next one's
  int32_t R;                             // rotary elements of a head; the table has R / 2 pairs a row
  int32_t chunks, span;                  // warps to a token, head groups to a warp
};

enum { kNoTurn = 0, kHalves = 1, kPairs = 2 };
constexpr int kRotaryThreads = 128;
constexpr int kGroupsAhead = 2;  // head groups whose words a lane asks for before it stores the first

// four neighbouring pairs of a 16-byte chunk, as rotate8 rounds
__device__ __forceinline__ uint4 rotate_pairs(const uint4& w, const float* c, const float* s) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x1 = __uint_as_float(in[j] << 16), x2 = __uint_as_float(in[j] & 0xffff0000u);
    const float y1 = __fsub_rn(__fmul_rn(x1, c[j]), __fmul_rn(x2, s[j]));
    const float y2 = __fadd_rn(__fmul_rn(x2, c[j]), __fmul_rn(x1, s[j]));
    out[j] = static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(y1))) |
             (static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(y2))) << 16);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

template <int D, int Turn>
__global__ void __launch_bounds__(kRotaryThreads) append_rotary_kernel(const __grid_constant__ RotaryArgs args) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const AppendArgs& a = args.a;
  constexpr int LPH = D / 16, HPW = 32 / LPH;  // lanes to a head, heads at a time
  const int heads = a.H_q + 2 * a.H_kv, groups = (heads + HPW - 1) / HPW;
  const int lane = threadIdx.x & 31, part = lane % LPH;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kRotaryThreads + threadIdx.x) >> 5;
  const int t = static_cast<int>(w / args.chunks);
  if (t >= a.T) return;
  const int g0 = static_cast<int>(w % args.chunks) * args.span, g1 = min(groups, g0 + args.span);
  const int slot = __ldg(a.slot_mapping + t);
  const bool slot_ok = slot >= 0 && static_cast<int64_t>(slot) < a.n_slots;
  if (!slot_ok && slot != -1 && a.status && lane == 0) atomicOr(a.status, MS_STATUS_BAD_SLOT);  // -1: no write
  // the lane's chunks, and whether they turn
  const int R = args.R, turning = R >> 4;
  const bool first_half = Turn != kHalves || part < turning;
  const int ia = Turn != kHalves ? part * 8 : first_half ? part * 8 : R + (part - turning) * 8;
  const int ib = Turn != kHalves ? D / 2 + part * 8 : first_half ? ia + (R >> 1) : ia + ((D - R) >> 1);
  const bool turn_a = Turn == kHalves ? first_half : Turn == kPairs && ia < R;
  const bool turn_b = Turn == kHalves ? first_half : Turn == kPairs && ib < R;
  float c[8], s[8];
  if constexpr (Turn != kNoTurn) {
    const int pos = __ldg(a.positions + t);
    // a token at a position outside the table writes nothing: no q_rot, no K, no V
    if (pos < 0 || pos >= a.max_pos) {
      if (a.status && lane == 0) atomicOr(a.status, MS_STATUS_BAD_POSITION);
      return;
    }
    const float* ct = a.cos_tab + static_cast<int64_t>(pos) * (R >> 1);
    const float* st = a.sin_tab + static_cast<int64_t>(pos) * (R >> 1);
    const int pa = Turn == kHalves ? part * 8 : ia >> 1, pb = Turn == kHalves ? part * 8 + 4 : ib >> 1;
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = s[j] = 0.f;
    if (turn_a) {
      const float4 c0 = __ldg(reinterpret_cast<const float4*>(ct + pa)), s0 = __ldg(reinterpret_cast<const float4*>(st + pa));
      c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
      s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
    }
    if (turn_b) {
      const float4 c1 = __ldg(reinterpret_cast<const float4*>(ct + pb)), s1 = __ldg(reinterpret_cast<const float4*>(st + pb));
      c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
      s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    }
  }
  const int64_t cell = slot_ok ? (static_cast<int64_t>(slot >> 4) * a.H_kv * 16 + (slot & 15)) * D : 0;  // of KV head 0
  const auto skipped = [&](int h) { return h >= heads || (h >= a.H_q && !slot_ok); };
  for (int g = g0; g < g1; g += kGroupsAhead) {
    uint4 xa[kGroupsAhead], xb[kGroupsAhead];
#pragma unroll
    for (int u = 0; u < kGroupsAhead; ++u) {
      const int h = (g + u) * HPW + lane / LPH;
      if (g + u >= g1 || h >= heads) continue;
      const __nv_bfloat16* src = h < a.H_q            ? a.q + t * args.q_stride + h * D
                                 : h < a.H_q + a.H_kv ? a.k + t * args.k_stride + (h - a.H_q) * D
                                                      : a.v + t * args.v_stride + (h - a.H_q - a.H_kv) * D;
      xa[u] = *reinterpret_cast<const uint4*>(src + ia);  // q_rot may be q: a lane reads its words before it writes them
      xb[u] = *reinterpret_cast<const uint4*>(src + ib);
    }
#pragma unroll
    for (int u = 0; u < kGroupsAhead; ++u) {
      const int h = (g + u) * HPW + lane / LPH;
      if (g + u >= g1 || skipped(h)) continue;
      __nv_bfloat16* dst;
      if (h < a.H_q) {
        dst = a.q_rot + (static_cast<int64_t>(t) * a.H_q + h) * D;
      } else if (h < a.H_q + a.H_kv) {
        dst = a.k_cache + cell + static_cast<int64_t>(h - a.H_q) * 16 * D;
      } else {
        dst = a.v_cache + cell + static_cast<int64_t>(h - a.H_q - a.H_kv) * 16 * D;
      }
      if (h < a.H_q + a.H_kv) {
        if constexpr (Turn == kHalves) {
          if (turn_a) {
            uint4 ya, yb;
            rotate8(xa[u], xb[u], c, s, ya, yb);
            xa[u] = ya;
            xb[u] = yb;
          }
        } else if constexpr (Turn == kPairs) {
          if (turn_a) xa[u] = rotate_pairs(xa[u], c, s);
          if (turn_b) xb[u] = rotate_pairs(xb[u], c + 4, s + 4);
        }
      }
      *reinterpret_cast<uint4*>(dst + ia) = xa[u];
      *reinterpret_cast<uint4*>(dst + ib) = xb[u];
    }
  }
}

}  // namespace

extern "C" MS_API int ms_rotary_frequencies(int32_t rotary_dim, double base, const ms_rotary_scaling* scaling, double* freq,
                                            double* amplitude) {
  const int R = rotary_dim;
  if (freq == nullptr || amplitude == nullptr || R < 2 || R % 2 != 0 || R > 2 * kMaxPairs || !(base > 0.0) ||
      !std::isfinite(base))
    return MS_ERR_ARG;
  const int kind = scaling != nullptr ? scaling->kind : MS_ROTARY_PLAIN;
  double s = 1.0, n = 1.0, low = 0.0, high = 0.0;
  if (kind != MS_ROTARY_PLAIN) {
    s = scaling->factor;
    if (kind < MS_ROTARY_LINEAR || kind > MS_ROTARY_RAMP || !(s > 0.0) || !std::isfinite(s)) return MS_ERR_ARG;
    if (kind == MS_ROTARY_BASE && R < 4) return MS_ERR_ARG;
    if (kind == MS_ROTARY_BANDS || kind == MS_ROTARY_RAMP) {
      n = scaling->original_len;
      low = scaling->low;
      high = scaling->high;
      if (!(n >= 1.0) || !(low > 0.0) || !(high > low) || !std::isfinite(high)) return MS_ERR_ARG;
      if (kind == MS_ROTARY_RAMP && (base == 1.0 || !(scaling->amplitude >= 0.0) || !std::isfinite(scaling->amplitude)))
        return MS_ERR_ARG;
    }
  }
  if (kind == MS_ROTARY_BASE) base *= std::pow(s, R / (R - 2.0));
  if (!(base > 0.0) || !std::isfinite(base)) return MS_ERR_ARG;
  double lo = 0.0, hi = 0.0;
  if (kind == MS_ROTARY_RAMP) {
    lo = std::fmax(std::floor(pair_of_turns(high, n, base, R)), 0.0);
    hi = std::fmax(std::fmin(std::ceil(pair_of_turns(low, n, base, R)), R - 1.0), lo);
    if (hi == lo) hi += 0.001;
  }
  double amp = 1.0, scaled[kMaxPairs];
  if (kind == MS_ROTARY_RAMP) amp = scaling->amplitude > 0.0 ? scaling->amplitude : s > 1.0 ? 0.1 * std::log(s) + 1.0 : 1.0;
  for (int i = 0; i < R / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / R);
    double g = f;
    if (kind == MS_ROTARY_LINEAR) {
      g = f / s;
    } else if (kind == MS_ROTARY_BANDS) {
      const double keep = std::fmin(1.0, std::fmax(0.0, (n * f / kTwoPi - low) / (high - low)));
      g = (1.0 - keep) * (f / s) + keep * f;
    } else if (kind == MS_ROTARY_RAMP) {
      const double stretch = std::fmin(1.0, std::fmax(0.0, (i - lo) / (hi - lo)));
      g = stretch * (f / s) + (1.0 - stretch) * f;
    }
    if (!std::isfinite(g)) return MS_ERR_ARG;
    scaled[i] = g;
  }
  for (int i = 0; i < R / 2; ++i) freq[i] = scaled[i];
  *amplitude = amp;
  return MS_OK;
}

extern "C" MS_API int ms_rotary_table_device(const double* freq, int32_t pairs, double amplitude, int32_t first_pos, int32_t n,
                                             float* cos_tab, float* sin_tab, ms_stream_t stream) {
  if (freq == nullptr || pairs < 4 || pairs % 4 != 0 || pairs > kMaxPairs || first_pos < 0 || n < 0 ||
      static_cast<int64_t>(first_pos) + n > (int64_t{1} << 31) || !(amplitude == 0.0 || (std::fabs(amplitude) >= 0x1p-40 && std::fabs(amplitude) <= 0x1p40)))
    return MS_ERR_ARG;
  for (int i = 0; i < pairs; ++i)
    if (!(std::fabs(freq[i]) <= 1024.0)) return MS_ERR_ARG;
  if (n == 0) return MS_OK;
  const auto al16 = [](const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al16(cos_tab) || !al16(sin_tab)) return MS_ERR_ARG;
  const int sms = ms_num_sms();
  if (sms <= 0) return MS_ERR_CUDA;
  TableArgs a;
  for (int i = 0; i < kMaxPairs; ++i) a.turns[i] = i < pairs ? turns_fixed(freq[i]) : 0;
  a.cos_tab = cos_tab;
  a.sin_tab = sin_tab;
  a.first = first_pos;
  a.n = n;
  a.half = pairs;
  const auto times = [&](double coefficient) { return static_cast<float>(amplitude * coefficient); };
  a.m.hi = times(1.0);
  a.m.lo = static_cast<float>(amplitude - static_cast<double>(a.m.hi));
  a.m.s3 = times(-1.0 / 6.0);
  a.m.s5 = times(1.0 / 120.0);
  a.m.s7 = times(-1.0 / 5040.0);
  a.m.s9 = times(1.0 / 362880.0);
  a.m.c2 = -0.5f * a.m.hi;  // exactly: what c_hi leaves out is taken from it
  a.m.c4 = times(1.0 / 24.0);
  a.m.c6 = times(-1.0 / 720.0);
  a.m.c8 = times(1.0 / 40320.0);
  a.m.c10 = times(-1.0 / 3628800.0);
  const int per_block = 256 / (pairs / 4);
  const int64_t need = (static_cast<int64_t>(n) + per_block - 1) / per_block, most = static_cast<int64_t>(sms) * 4;
  const unsigned blocks = static_cast<unsigned>(need < most ? need : most);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (amplitude == 1.0)
    rotary_table_kernel<false><<<blocks, 256, 0, st>>>(a);
  else
    rotary_table_kernel<true><<<blocks, 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}

extern "C" MS_API int ms_kv_append_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                          int64_t v_stride, const int32_t* positions, const int32_t* slot_mapping, int32_t T,
                                          const float* cos_tab, const float* sin_tab, int32_t max_pos, int32_t rotary_dim,
                                          int32_t interleaved, void* k_cache, void* v_cache, int32_t num_pages, void* q_rot,
                                          int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size, int32_t* dev_status,
                                          ms_stream_t stream) {
  const int R = rotary_dim;
  if (T < 0 || H_q < 0 || H_kv < 1 || (D != 64 && D != 128) || page_size != 16 || num_pages < 0 || R < 0 || R > D ||
      R % 16 != 0 || (interleaved != 0 && interleaved != 1) || (R > 0 && max_pos < 1) || H_q > 65536 || H_kv > 65536)
    return MS_ERR_ARG;
  // a token's heads lie side by side; tokens must not overlap and start on 16 bytes
  const auto stride_ok = [](int64_t s, int64_t row) { return s >= row && s % 8 == 0 && s <= (int64_t{1} << 40); };
  if ((H_q > 0 && !stride_ok(q_stride, static_cast<int64_t>(H_q) * D)) || !stride_ok(k_stride, static_cast<int64_t>(H_kv) * D) ||
      !stride_ok(v_stride, static_cast<int64_t>(H_kv) * D))
    return MS_ERR_ARG;
  if (T == 0) return MS_OK;
  const auto al16 = [](const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al16(k) || !al16(v) || !al16(k_cache) || !al16(v_cache) || slot_mapping == nullptr ||
      (H_q > 0 && (!al16(q) || !al16(q_rot))) || (R > 0 && (positions == nullptr || !al16(cos_tab) || !al16(sin_tab))))
    return MS_ERR_ARG;
  // in place only row on row: with gaps between the tokens' rows q_rot would lie over other rows of q
  if (H_q > 0 && q == q_rot && q_stride != static_cast<int64_t>(H_q) * D) return MS_ERR_ARG;
  RotaryArgs args;
  AppendArgs& a = args.a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.positions = positions;
  a.slot_mapping = slot_mapping;
  a.cos_tab = cos_tab;
  a.sin_tab = sin_tab;
  a.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  a.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  a.q_rot = static_cast<__nv_bfloat16*>(q_rot);
  a.status = dev_status;
  a.n_slots = static_cast<int64_t>(num_pages) * 16;
  a.T = T;
  a.H_q = H_q;
  a.H_kv = H_kv;
  a.D = D;
  a.max_pos = max_pos;
  a.page = 16;
  args.q_stride = q_stride;
  args.k_stride = k_stride;
  args.v_stride = v_stride;
  args.R = R;
  const int sms = ms_num_sms();
  if (sms <= 0) return MS_ERR_CUDA;
  // a warp to a token, or several where the tokens alone would not fill the SMs with 32 warps
  const int per_group = D == 128 ? 4 : 8, groups = (H_q + 2 * H_kv + per_group - 1) / per_group;
  int64_t chunks = (static_cast<int64_t>(sms) * 32 + T - 1) / T;
  chunks = chunks < 1 ? 1 : chunks > groups ? groups : chunks;
  args.span = static_cast<int32_t>((groups + chunks - 1) / chunks);
  args.chunks = (groups + args.span - 1) / args.span;
  const int64_t warps = static_cast<int64_t>(T) * args.chunks;
  const int64_t blocks64 = (warps + kRotaryThreads / 32 - 1) / (kRotaryThreads / 32);
  if (blocks64 > INT32_MAX) return MS_ERR_ARG;
  const unsigned blocks = static_cast<unsigned>(blocks64);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const auto kernel = D == 128 ? (R == 0        ? append_rotary_kernel<128, kNoTurn>
                                  : interleaved ? append_rotary_kernel<128, kPairs>
                                                : append_rotary_kernel<128, kHalves>)
                               : (R == 0        ? append_rotary_kernel<64, kNoTurn>
                                  : interleaved ? append_rotary_kernel<64, kPairs>
                                                : append_rotary_kernel<64, kHalves>);
  kernel<<<blocks, kRotaryThreads, 0, st>>>(args);
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}
