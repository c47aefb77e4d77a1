// The append into a 4-bit cache and the read-back of its rows.
//
// Append: rotary embedding at absolute positions (as in append_rope.cuh, the
// same rounding, so q_rot is bit for bit that of the bf16 append), then K and V
// rounded to 4 bits (q4.cuh) into the pages.  A warp takes heads of one token, 4
// at a time (8 at D = 64): a lane owns 8 consecutive element pairs (i, i + D/2)
// of a head and keeps the token's cosines and sines for them, which a thread per
// (token, head) would read again for every head.  The four lanes of a 32-element
// group exchange its largest magnitude, and pairs of lanes trade words so that
// each stores 8 contiguous bytes of a row.  It has to move (4 H_q + 6.25 H_kv) D bytes
// and 4 D of the tables a token.  8192 tokens, 32 / 8 heads, D = 128: 40 us, 4.8 TB/s,
// 0.71 of the measured copy rate, issue slots 62 % busy; about 32 KB are on their way
// to an SM (a lane's next 32 bytes), fewer than a round trip at the copy rate covers.
#include <cuda_runtime.h>

#include <cstdint>

#include "append_rope.cuh"
#include "mixed_step.h"
#include "q4.cuh"

namespace {

struct AppendQ4Args {
  AppendArgs a;  // k_cache and v_cache unused
  uint8_t* kv_cache;
  int32_t chunks;  // warps to a token
  int32_t span;    // head groups to a warp
};

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf16_lo(u[j]);
    x[2 * j + 1] = bf16_hi(u[j]);
  }
}

// One lane's 8 elements of a group -> their 8 nibbles in K order (elements 0, 2,
// 4, 6 in the low half, 1, 3, 5, 7 in the high half) and the group's scale, as
// bf16 bits.  `mask`: the four lanes of the group.  Magnitudes compare as 16-bit
// whole numbers, an infinity or a NaN above every finite one: a group that holds
// one is stored as zeros.
__device__ __forceinline__ uint32_t quantize8(const uint4& w, unsigned mask, uint32_t& scale, bool& finite) {
  const uint32_t m2 = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
  uint32_t m = max(m2 & 0xffffu, m2 >> 16);
  m = max(m, __shfl_xor_sync(mask, m, 1));
  m = max(m, __shfl_xor_sync(mask, m, 2));
  finite = m < 0x7f80u;
  const float s = finite ? q4_scale(__uint_as_float(m << 16)) : 0.f;
  scale = __float_as_uint(s) >> 16;  // five significant bits
  if (s == 0.f) return 0x88888888u;
  const float r = __frcp_rn(s);
  float x[8];
  unpack8(w, x);
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) word |= q4_nibble(x[e], r) << (4 * ((e & 1) * 4 + (e >> 1)));
  return word;
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_q4_kernel(AppendQ4Args args) {
  using Q = Q4<D>;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const AppendArgs& a = args.a;
  constexpr int half = D / 2, LPH = half / kAppendVec, HPW = 32 / LPH;  // lanes to a head, heads at a time
  const int heads = a.H_q + 2 * a.H_kv, groups = (heads + HPW - 1) / HPW;
  const int lane = threadIdx.x & 31, part = lane % LPH, i0 = part * kAppendVec;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x) >> 5;
  const int t = static_cast<int>(w / args.chunks);
  if (t >= a.T) return;
  const int g0 = static_cast<int>(w % args.chunks) * args.span, g1 = min(groups, g0 + args.span);
  const int pos = __ldg(a.positions + t), slot = __ldg(a.slot_mapping + t);
  const bool slot_ok = slot >= 0 && static_cast<int64_t>(slot) < a.n_slots;
  if (!slot_ok && slot != -1 && a.status && lane == 0) atomicOr(a.status, MS_STATUS_BAD_SLOT);  // -1: no write
  // a token at a position outside the table writes nothing: no q_rot, no K, no V
  if (pos < 0 || pos >= a.max_pos) {
    if (a.status && lane == 0) atomicOr(a.status, MS_STATUS_BAD_POSITION);
    return;
  }
  float c[kAppendVec], s[kAppendVec];
  {
    const float4* cp = reinterpret_cast<const float4*>(a.cos_tab + static_cast<int64_t>(pos) * half + i0);
    const float4* sp = reinterpret_cast<const float4*>(a.sin_tab + static_cast<int64_t>(pos) * half + i0);
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
    c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
  }
  const unsigned group_mask = 0xfu << (lane & 28), head_mask = (LPH == 8 ? 0xffu : 0xfu) << (lane & (32 - LPH));
  uint8_t* row0 = args.kv_cache;  // block of KV head 0 of the slot's page
  const int row = slot_ok ? slot % kQ4Page : 0;
  if (slot_ok) row0 += static_cast<int64_t>(slot / kQ4Page) * a.H_kv * Q::BYTES;
  // the lane's two 16-byte words of head h: q, then k, then v (zeros past the last head)
  auto load = [&](int h, uint4& xa, uint4& xb) {
    xa = xb = make_uint4(0, 0, 0, 0);
    if (h >= heads || (h >= a.H_q && !slot_ok)) return;
    const __nv_bfloat16* src = h < a.H_q              ? a.q + (static_cast<int64_t>(t) * a.H_q + h) * D
                               : h < a.H_q + a.H_kv ? a.k + (static_cast<int64_t>(t) * a.H_kv + h - a.H_q) * D
                                                    : a.v + (static_cast<int64_t>(t) * a.H_kv + h - a.H_q - a.H_kv) * D;
    xa = *reinterpret_cast<const uint4*>(src + i0);  // q_rot may be q: a lane reads its words before it writes them
    xb = *reinterpret_cast<const uint4*>(src + i0 + half);
  };
  uint4 xa, xb, na, nb;
  load(g0 * HPW + lane / LPH, xa, xb);
  for (int g = g0; g < g1; ++g, xa = na, xb = nb) {
    const int h = g * HPW + lane / LPH;
    if (g + 1 < g1) load(h + HPW, na, nb);
    if (h >= heads || (h >= a.H_q && !slot_ok)) continue;
    const bool is_v = h >= a.H_q + a.H_kv;
    if (!is_v) {
      uint4 ya, yb;
      rotate8(xa, xb, c, s, ya, yb);
      xa = ya;
      xb = yb;
    }
    if (h < a.H_q) {
      __nv_bfloat16* dst = a.q_rot + (static_cast<int64_t>(t) * a.H_q + h) * D;
      *reinterpret_cast<uint4*>(dst + i0) = xa;
      *reinterpret_cast<uint4*>(dst + i0 + half) = xb;
      continue;
    }
    uint32_t sa, sb;
    bool fa, fb;
    const uint32_t wa = quantize8(xa, group_mask, sa, fa), wb = quantize8(xb, group_mask, sb, fb);
    if (!(fa && fb) && a.status && (part & 3) == 0) atomicOr(a.status, MS_STATUS_NONFINITE);
    uint8_t* blk = row0 + (is_v ? h - a.H_q - a.H_kv : h - a.H_q) * Q::BYTES;
    // elements i0.. are in group p4 = part / 4 (0 at D = 64), those of the second half NG / 2 groups on;
    // with the lane of the other p4 a quarter's bytes are complete, and each of the two stores a half
    const int quarter = part & 3, p4 = part >> 2;
    uint32_t w0, w1;
    if (!is_v) {
      if constexpr (D == 128) {
        const uint32_t got = __shfl_xor_sync(head_mask, p4 == 0 ? wb : wa, 4);
        w0 = p4 == 0 ? wa : got;
        w1 = p4 == 0 ? got : wb;
      } else {
        w0 = wa;
        w1 = wb;
      }
    } else {
      const uint32_t even = join_halves(wa, wb, 0), odd = join_halves(wa, wb, 1);  // of the groups p4 and p4 + NG / 2
      if constexpr (D == 128) {
        const uint32_t got = __shfl_xor_sync(head_mask, p4 == 0 ? odd : even, 4);
        const uint32_t mine = p4 == 0 ? even : odd, first = p4 == 0 ? mine : got, second = p4 == 0 ? got : mine;
        w0 = join_halves(first, second, 0);  // groups 0 and 1
        w1 = join_halves(first, second, 1);  // groups 2 and 3
      } else {
        w0 = even;
        w1 = odd;
      }
    }
    *reinterpret_cast<uint2*>(blk + (is_v ? Q::V_OFF : 0) + row * Q::ROW + quarter * (Q::ROW / 4) + p4 * 8) = make_uint2(w0, w1);
    uint8_t* sc = blk + (is_v ? Q::VS_OFF : Q::KS_OFF) + row * Q::NG * 2;
    if constexpr (D == 128) {
      const uint32_t mine = sa | (sb << 16);  // groups p4 and p4 + 2
      const uint32_t got = __shfl_xor_sync(head_mask, mine, 4);
      if (part == 0) *reinterpret_cast<uint2*>(sc) = make_uint2(join_halves(mine, got, 0), join_halves(mine, got, 1));
    } else {
      if (part == 0) *reinterpret_cast<uint32_t*>(sc) = sa | (sb << 16);
    }
  }
}

struct ReadQ4Args {
  const uint8_t* kv_cache;
  const int32_t* slots;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int32_t* status;
  int64_t n_slots;
  int32_t n, H_kv;
};

// Eight nibbles in K order -> their bf16 values, elements in order.
__device__ __forceinline__ uint4 dequantize8(uint32_t word, uint32_t s2) {
  return make_uint4(q4_pair_times(word, 0, s2), q4_pair_times(word, 1, s2), q4_pair_times(word, 2, s2),
                    q4_pair_times(word, 3, s2));
}

// One thread per quarter of one (slot, KV head) row of K and of V: 8 elements
// of every group, whose codes are contiguous (16 bytes at D = 128).  HBM-bound:
// 6000 rows of 8 heads, D = 128, take 4.8 us in a replayed graph (31.5 MB: 4.7 us at
// the measured copy rate); fewer rows are a launch, 1.9 us there.
template <int D, typename Idx>
__global__ void __launch_bounds__(256) read_q4_kernel(ReadQ4Args a) {
  using Q = Q4<D>;
  constexpr int NG = Q::NG;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // launched while the kernel before it, an append, still runs
  const Idx total = static_cast<Idx>(a.n) * a.H_kv * 4;
  const Idx stride = static_cast<Idx>(gridDim.x) * 256;
  for (Idx u = static_cast<Idx>(blockIdx.x) * 256 + threadIdx.x; u < total; u += stride) {
    const int t = static_cast<int>(u & 3);
    const Idx rh = u >> 2;
    const int h = static_cast<int>(rh % a.H_kv);
    const int slot = __ldg(a.slots + rh / a.H_kv);
    uint32_t k[NG], v[NG], ks[NG / 2], vs[NG / 2];
    if (slot >= 0 && static_cast<int64_t>(slot) < a.n_slots) {
      const uint8_t* blk = a.kv_cache + (static_cast<int64_t>(slot / kQ4Page) * a.H_kv + h) * Q::BYTES;
      const int row = slot % kQ4Page;
      ldg_words<NG>(blk + row * Q::ROW + t * 4 * NG, k);
      ldg_words<NG>(blk + Q::V_OFF + row * Q::ROW + t * 4 * NG, v);
      ldg_words<NG / 2>(blk + Q::KS_OFF + row * NG * 2, ks);
      ldg_words<NG / 2>(blk + Q::VS_OFF + row * NG * 2, vs);
    } else {
      if (slot != -1 && a.status && t == 0) atomicOr(a.status, MS_STATUS_BAD_SLOT);
#pragma unroll
      for (int g = 0; g < NG; ++g) k[g] = v[g] = 0u;
#pragma unroll
      for (int g = 0; g < NG / 2; ++g) ks[g] = vs[g] = 0u;
    }
    const int64_t base = static_cast<int64_t>(rh) * D + 8 * t;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const uint32_t sel = g & 1 ? 0x3232 : 0x1010;
      *reinterpret_cast<uint4*>(a.k_out + base + 32 * g) = dequantize8(k[g], __byte_perm(ks[g >> 1], 0, sel));
      // V's even elements lie below its odd ones in each half of the quarter's bytes
      const uint32_t w = join_halves(v[g >> 1], v[NG / 2 + (g >> 1)], g & 1);
      *reinterpret_cast<uint4*>(a.v_out + base + 32 * g) = dequantize8(w, __byte_perm(vs[g >> 1], 0, sel));
    }
  }
}

}  // namespace

extern "C" MS_API int64_t ms_q4_block_bytes(int32_t D) { return D == 64 || D == 128 ? q4_block_bytes(D) : 0; }

extern "C" MS_API int ms_kv_append_rope_q4(const void* q, const void* k, const void* v, const int32_t* positions,
                                           const int32_t* slot_mapping, int32_t T, const float* cos_tab,
                                           const float* sin_tab, int32_t max_pos, void* kv_cache, int32_t num_pages,
                                           void* q_rot, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
                                           int32_t* dev_status, ms_stream_t stream) {
  AppendQ4Args args;
  int64_t units = 0;
  const int rc = append_setup(q, k, v, positions, slot_mapping, T, cos_tab, sin_tab, max_pos, kv_cache, kv_cache,
                              num_pages, q_rot, H_q, H_kv, D, page_size, dev_status, &args.a, &units);
  if (rc != MS_OK || units == 0) return rc;
  args.kv_cache = static_cast<uint8_t*>(kv_cache);
  const int sms = ms_num_sms();
  if (sms <= 0) return MS_ERR_CUDA;
  // a warp to a token, or several where the tokens alone would not fill the SMs with 32 warps (8192
  // tokens, 32 / 8 heads, with the read-back, as the kernel was then: 51 us a warp to a token, 55 us with three)
  const int per_group = D == 128 ? 4 : 8, groups = (H_q + 2 * H_kv + per_group - 1) / per_group;
  int64_t chunks = (static_cast<int64_t>(sms) * 32 + T - 1) / T;
  chunks = chunks < 1 ? 1 : chunks > groups ? groups : chunks;
  args.span = static_cast<int32_t>((groups + chunks - 1) / chunks);
  args.chunks = (groups + args.span - 1) / args.span;
  const int64_t warps = static_cast<int64_t>(T) * args.chunks;
  const int64_t blocks64 = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  if (blocks64 > INT32_MAX) return MS_ERR_ARG;
  const unsigned blocks = static_cast<unsigned>(blocks64);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128)
    append_q4_kernel<128><<<blocks, kAppendThreads, 0, st>>>(args);
  else
    append_q4_kernel<64><<<blocks, kAppendThreads, 0, st>>>(args);
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}

extern "C" MS_API int ms_kv_read_q4(const void* kv_cache, int32_t num_pages, const int32_t* slots, int32_t n, void* k_out,
                                    void* v_out, int32_t H_kv, int32_t D, int32_t page_size, int32_t* dev_status,
                                    ms_stream_t stream) {
  if (num_pages < 0 || n < 0 || H_kv < 1 || (D != 64 && D != 128) || page_size != kQ4Page) return MS_ERR_ARG;
  if (n == 0) return MS_OK;
  const auto al16 = [](const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al16(kv_cache) || !al16(k_out) || !al16(v_out) || slots == nullptr) return MS_ERR_ARG;
  ReadQ4Args a;
  a.kv_cache = static_cast<const uint8_t*>(kv_cache);
  a.slots = slots;
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.status = dev_status;
  a.n_slots = static_cast<int64_t>(num_pages) * kQ4Page;
  a.n = n;
  a.H_kv = H_kv;
  const int64_t units = static_cast<int64_t>(n) * H_kv * 4;
  const int sms = ms_num_sms();
  if (sms <= 0) return MS_ERR_CUDA;
  const unsigned blocks = static_cast<unsigned>(append_blocks(units, sms));
  const bool small = units + static_cast<int64_t>(blocks) * 256 < (int64_t{1} << 31);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const auto kernel = D == 128 ? (small ? read_q4_kernel<128, uint32_t> : read_q4_kernel<128, int64_t>)
                               : (small ? read_q4_kernel<64, uint32_t> : read_q4_kernel<64, int64_t>);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess && cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}
