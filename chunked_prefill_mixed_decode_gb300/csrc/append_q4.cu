// The append into a 4-bit cache and the read-back of its rows.
//
// Append: rotary embedding at absolute positions (as in append_rope.cuh, the
// same rounding, so q_rot is bit for bit that of the bf16 append), then K and V
// rounded to 4 bits (q4.cuh) into the pages.  One thread owns 8 consecutive
// element pairs (i, i + D/2) of one (token, head) row; the four threads of a
// 32-element group exchange its largest magnitude by shuffles.
#include <cuda_runtime.h>

#include <cstdint>

#include "append_rope.cuh"
#include "mixed_step.h"
#include "q4.cuh"

namespace {

struct AppendQ4Args {
  AppendArgs a;  // k_cache and v_cache unused
  uint8_t* kv_cache;
};

__device__ __forceinline__ void unpack8(const uint4& w, float* x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = bf16_lo(u[j]);
    x[2 * j + 1] = bf16_hi(u[j]);
  }
}

// One thread's 8 elements of a group -> their 8 nibbles in K order (elements
// 0, 2, 4, 6 in the low half, 1, 3, 5, 7 in the high half) and the group's
// scale.  `mask`: the four lanes of the group.  A group that holds an infinity
// or a NaN is stored as zeros.
__device__ __forceinline__ uint32_t quantize8(const uint4& w, unsigned mask, float& scale, bool& finite) {
  float x[8];
  unpack8(w, x);
  float a = 0.f;
  finite = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    a = fmaxf(a, fabsf(x[j]));
    finite = finite && isfinite(x[j]);
  }
  a = fmaxf(a, __shfl_xor_sync(mask, a, 1));
  a = fmaxf(a, __shfl_xor_sync(mask, a, 2));
  finite = __all_sync(mask, finite);
  scale = finite ? q4_scale(a) : 0.f;
  uint32_t word = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) word |= q4_nibble(finite ? x[e] : 0.f, scale) << (4 * ((e & 1) * 4 + (e >> 1)));
  return word;
}

template <int D>
__device__ __forceinline__ void store_group_part(uint8_t* blk, int row, bool is_v, int d0, uint32_t word, float scale) {
  using Q = Q4<D>;
  const int g = d0 / kQ4Group, t = (d0 % kQ4Group) / 8;
  if (!is_v) {
    *reinterpret_cast<uint32_t*>(blk + row * Q::ROW + (t * Q::NG + g) * 4) = word;
  } else {
    uint8_t* dst = blk + Q::V_OFF + row * Q::ROW + (2 * t * Q::NG + g) * 2;
    *reinterpret_cast<uint16_t*>(dst) = static_cast<uint16_t>(word);
    *reinterpret_cast<uint16_t*>(dst + 2 * Q::NG) = static_cast<uint16_t>(word >> 16);
  }
  if (t == 0)
    *reinterpret_cast<__nv_bfloat16*>(blk + (is_v ? Q::VS_OFF : Q::KS_OFF) + (row * Q::NG + g) * 2) =
        __float2bfloat16_rn(scale);
}

template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_q4_kernel(AppendQ4Args args) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const AppendArgs& a = args.a;
  constexpr int half = D / 2, per_row = half / kAppendVec;
  const int heads = a.H_q + 2 * a.H_kv;
  const int64_t total = static_cast<int64_t>(a.T) * heads * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kAppendThreads;
  const unsigned mask = 0xfu << (threadIdx.x & 28);
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * kAppendThreads + threadIdx.x; g < total; g += stride) {
    const int part = static_cast<int>(g % per_row);
    const int64_t rh = g / per_row;
    const int h = static_cast<int>(rh % heads);
    const int t = static_cast<int>(rh / heads);
    const int i0 = part * kAppendVec;
    const int pos = __ldg(a.positions + t);
    const int slot = __ldg(a.slot_mapping + t);
    if (h >= a.H_q) {
      if (slot == -1) continue;
      if (slot < 0 || static_cast<int64_t>(slot) >= a.n_slots) {
        if (a.status && part == 0) atomicOr(a.status, MS_STATUS_BAD_SLOT);
        continue;
      }
    }
    if (pos < 0 || pos >= a.max_pos) {
      if (a.status && part == 0) atomicOr(a.status, MS_STATUS_BAD_POSITION);
      continue;
    }
    const bool is_v = h >= a.H_q + a.H_kv;
    const int hk = is_v ? h - a.H_q - a.H_kv : h - a.H_q;
    const __nv_bfloat16* src = h < a.H_q ? a.q + (static_cast<int64_t>(t) * a.H_q + h) * D
                                         : (is_v ? a.v : a.k) + (static_cast<int64_t>(t) * a.H_kv + hk) * D;
    uint4 xa = *reinterpret_cast<const uint4*>(src + i0);
    uint4 xb = *reinterpret_cast<const uint4*>(src + i0 + half);
    if (!is_v) {
      float c[kAppendVec], s[kAppendVec];
      const float4* cp = reinterpret_cast<const float4*>(a.cos_tab + static_cast<int64_t>(pos) * half + i0);
      const float4* sp = reinterpret_cast<const float4*>(a.sin_tab + static_cast<int64_t>(pos) * half + i0);
      const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(sp), s1 = __ldg(sp + 1);
      c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w; c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
      s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w; s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
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
    float sa, sb;
    bool fa, fb;
    const uint32_t wa = quantize8(xa, mask, sa, fa), wb = quantize8(xb, mask, sb, fb);
    if (!(fa && fb) && a.status && (part & 3) == 0) atomicOr(a.status, MS_STATUS_NONFINITE);
    uint8_t* blk = args.kv_cache + (static_cast<int64_t>(slot / kQ4Page) * a.H_kv + hk) * Q4<D>::BYTES;
    store_group_part<D>(blk, slot % kQ4Page, is_v, i0, wa, sa);
    store_group_part<D>(blk, slot % kQ4Page, is_v, i0 + half, wb, sb);
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
__device__ __forceinline__ uint4 dequantize8(uint32_t word, float s) {
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = static_cast<float>(static_cast<int>((word >> (4 * i)) & 15u) - 8) * s;
    const float hi = static_cast<float>(static_cast<int>((word >> (16 + 4 * i)) & 15u) - 8) * s;
    const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    out[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}

// One thread per 8 elements of one (slot, KV head) row of K and of V.
template <int D>
__global__ void __launch_bounds__(256) read_q4_kernel(ReadQ4Args a) {
  using Q = Q4<D>;
  constexpr int per_row = D / 8;
  const int64_t total = static_cast<int64_t>(a.n) * a.H_kv * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; u < total; u += stride) {
    const int part = static_cast<int>(u % per_row);
    const int64_t rh = u / per_row;
    const int h = static_cast<int>(rh % a.H_kv);
    const int64_t r = rh / a.H_kv;
    const int slot = __ldg(a.slots + r);
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (slot >= 0 && static_cast<int64_t>(slot) < a.n_slots) {
      const uint8_t* blk = a.kv_cache + (static_cast<int64_t>(slot / kQ4Page) * a.H_kv + h) * Q::BYTES;
      const int row = slot % kQ4Page, g = part / 4, t = part % 4;
      const uint32_t kw = *reinterpret_cast<const uint32_t*>(blk + row * Q::ROW + (t * Q::NG + g) * 4);
      const uint8_t* vp = blk + Q::V_OFF + row * Q::ROW + (2 * t * Q::NG + g) * 2;
      const uint32_t vw = *reinterpret_cast<const uint16_t*>(vp) |
                          (static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(vp + 2 * Q::NG)) << 16);
      const float ks = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(blk + Q::KS_OFF + (row * Q::NG + g) * 2));
      const float vs = __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(blk + Q::VS_OFF + (row * Q::NG + g) * 2));
      k = dequantize8(kw, ks);
      v = dequantize8(vw, vs);
    } else if (slot != -1 && a.status && part == 0) {
      atomicOr(a.status, MS_STATUS_BAD_SLOT);
    }
    const int64_t base = (r * a.H_kv + h) * D + 8 * part;
    *reinterpret_cast<uint4*>(a.k_out + base) = k;
    *reinterpret_cast<uint4*>(a.v_out + base) = v;
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
  const unsigned blocks = static_cast<unsigned>(append_blocks(units, 152));
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
  const unsigned blocks = static_cast<unsigned>(append_blocks(static_cast<int64_t>(n) * H_kv * (D / 8), 152));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (D == 128)
    read_q4_kernel<128><<<blocks, 256, 0, st>>>(a);
  else
    read_q4_kernel<64><<<blocks, 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}
