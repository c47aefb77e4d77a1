// Mixed-batch attention over a paged 4-bit K/V cache: the plainest kernel.
// One warp per (packed token, KV head) walks its keys page by page: lane l
// takes key l % 16 of the page and half l / 16 of the head dim for the scores
// of the G query heads, the running maximum and sum follow in fp32, and every
// lane owns D / 32 columns of the output.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "mixed_step.h"
#include "q4.cuh"

namespace {

struct Q4AttnArgs {
  const __nv_bfloat16* q_rot;
  const uint8_t* kv;
  const int32_t* cu;
  const int32_t* q_start;
  const int32_t* ctx;
  const int32_t* bt;
  const int32_t* bt_off;
  __nv_bfloat16* out;
  int32_t* status;
  int64_t bt_len;
  int32_t bt_stride, num_rows, num_tokens, num_pages, H_q, H_kv;
  float scale_log2;
};

template <int D>
__device__ __forceinline__ float q4_value(const uint8_t* blk, int row, int d, bool is_v) {
  using Q = Q4<D>;
  const int g = d / 32, t = (d % 32) / 8, e = d % 8;
  const int nib = is_v ? ((2 * t + (e & 1)) * Q::NG + g) * 4 + e / 2 : (t * Q::NG + g) * 8 + (e & 1) * 4 + e / 2;
  const int b = blk[(is_v ? Q::V_OFF : 0) + row * Q::ROW + nib / 2];
  const float s = __bfloat162float(
      *reinterpret_cast<const __nv_bfloat16*>(blk + (is_v ? Q::VS_OFF : Q::KS_OFF) + (row * Q::NG + g) * 2));
  return static_cast<float>(((b >> (4 * (nib & 1))) & 15) - 8) * s;
}

template <int D, int G>
__global__ void __launch_bounds__(128) attention_q4_simple(Q4AttnArgs a) {
  constexpr int EPL = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) >> 5;
  if (w >= static_cast<int64_t>(a.num_tokens) * a.H_kv) return;
  const int t = static_cast<int>(w / a.H_kv), hk = static_cast<int>(w % a.H_kv);
  int row = -1;
  for (int s = lane; s < a.num_rows; s += 32)
    if (a.cu[s] <= t && t < a.cu[s + 1]) row = s;
  row = __reduce_max_sync(0xffffffffu, row);
  if (row < 0) return;
  const int64_t c = a.q_start[row], d = static_cast<int64_t>(a.cu[row + 1]) - a.cu[row], n_ctx = a.ctx[row];
  const int64_t o0 = a.bt_off != nullptr ? a.bt_off[row] : static_cast<int64_t>(row) * a.bt_stride;
  const int64_t len = a.bt_off != nullptr ? a.bt_off[row + 1] - o0 : a.bt_stride;
  if (a.cu[row] < 0 || a.cu[row + 1] > a.num_tokens || c < 0 || n_ctx != c + d || (n_ctx + 15) / 16 > len || o0 < 0 ||
      o0 + len > a.bt_len) {
    if (lane == 0) atomicOr(a.status, MS_STATUS_BAD_META);
    return;
  }
  const int pos = static_cast<int>(c + t - a.cu[row]);
  float m[G], l[G], acc[G][EPL];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    for (int e = 0; e < EPL; ++e) acc[h][e] = 0.f;
  }
  const __nv_bfloat16* q = a.q_rot + (static_cast<int64_t>(t) * a.H_q + hk * G) * D;
  for (int k0 = 0; k0 <= pos; k0 += 16) {
    int phys = a.bt[o0 + k0 / 16];
    if (phys < 0 || phys >= a.num_pages) {
      if (lane == 0) atomicOr(a.status, MS_STATUS_BAD_PAGE);
      phys = 0;
    }
    const uint8_t* blk = a.kv + (static_cast<int64_t>(phys) * a.H_kv + hk) * Q4<D>::BYTES;
    const int key = lane & 15, half = lane >> 4;
    float s[G];
    for (int h = 0; h < G; ++h) s[h] = 0.f;
    for (int i = half * (D / 2); i < (half + 1) * (D / 2); ++i) {
      const float kv = q4_value<D>(blk, key, i, false);
      for (int h = 0; h < G; ++h) s[h] += __bfloat162float(q[h * D + i]) * kv;
    }
    const int nv = min(16, pos + 1 - k0);
    for (int h = 0; h < G; ++h) {
      s[h] += __shfl_xor_sync(0xffffffffu, s[h], 16);
      s[h] = key < nv ? s[h] * a.scale_log2 : -INFINITY;
      float mx = s[h];
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[h], mx), al = exp2f(m[h] - mn);
      m[h] = mn;
      s[h] = exp2f(s[h] - mn);
      float sum = s[h];
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      l[h] = l[h] * al + sum;
      for (int e = 0; e < EPL; ++e) acc[h][e] *= al;
    }
    for (int j = 0; j < nv; ++j)
      for (int e = 0; e < EPL; ++e) {
        const float v = q4_value<D>(blk, j, lane * EPL + e, true);
        for (int h = 0; h < G; ++h) acc[h][e] += __shfl_sync(0xffffffffu, s[h], j) * v;
      }
  }
  for (int h = 0; h < G; ++h)
    for (int e = 0; e < EPL; ++e)
      a.out[(static_cast<int64_t>(t) * a.H_q + hk * G + h) * D + lane * EPL + e] = __float2bfloat16_rn(acc[h][e] / l[h]);
}

}  // namespace

extern "C" MS_API int ms_mixed_step_attention_q4(const void* q_rot, const void* kv_cache, int32_t num_pages,
                                                 const int32_t* cu_seqlens_q, const int32_t* q_start_pos,
                                                 const int32_t* context_lens, const int32_t* block_tables,
                                                 const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride,
                                                 int32_t num_rows, int32_t num_tokens, int64_t context_total, int32_t H_q,
                                                 int32_t H_kv, int32_t D, int32_t page_size, float scale, void* out,
                                                 void* workspace, size_t ws_bytes, ms_stream_t stream) {
  if (num_rows < 0 || num_tokens < 0 || context_total < 0 || H_q < 1 || H_kv < 1 || H_q % H_kv != 0 ||
      (D != 64 && D != 128) || page_size != 16 || bt_stride < 0 || bt_len < 0 || num_pages < 0 || !(scale > 0.f))
    return MS_ERR_ARG;
  if (num_rows == 0 || num_tokens == 0) return MS_OK;
  const int G = H_q / H_kv;
  if (!q_rot || !kv_cache || !cu_seqlens_q || !q_start_pos || !context_lens || !block_tables || !out || !workspace ||
      num_pages < 1 || (bt_offsets ? bt_len < 1 : bt_stride < 1))
    return MS_ERR_ARG;
  const auto al16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!al16(q_rot) || !al16(kv_cache) || !al16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      num_rows > 8192 || num_tokens > (1 << 21))
    return MS_ERR_ARG;
  if (ws_bytes < ms_attention_workspace_size(num_rows, num_tokens, context_total, H_q, H_kv, D)) return MS_ERR_ARG;
  Q4AttnArgs a{static_cast<const __nv_bfloat16*>(q_rot), static_cast<const uint8_t*>(kv_cache), cu_seqlens_q, q_start_pos,
               context_lens, block_tables, bt_offsets, static_cast<__nv_bfloat16*>(out), static_cast<int32_t*>(workspace),
               bt_offsets ? bt_len : static_cast<int64_t>(num_rows) * bt_stride, bt_stride, num_rows, num_tokens, num_pages,
               H_q, H_kv, scale * 1.4426950408889634f};
  const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(num_tokens) * H_kv + 3) / 4);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  switch (D * 100 + G) {
    case 6401: attention_q4_simple<64, 1><<<blocks, 128, 0, st>>>(a); break;
    case 6402: attention_q4_simple<64, 2><<<blocks, 128, 0, st>>>(a); break;
    case 6404: attention_q4_simple<64, 4><<<blocks, 128, 0, st>>>(a); break;
    case 6408: attention_q4_simple<64, 8><<<blocks, 128, 0, st>>>(a); break;
    case 12801: attention_q4_simple<128, 1><<<blocks, 128, 0, st>>>(a); break;
    case 12802: attention_q4_simple<128, 2><<<blocks, 128, 0, st>>>(a); break;
    case 12804: attention_q4_simple<128, 4><<<blocks, 128, 0, st>>>(a); break;
    case 12808: attention_q4_simple<128, 8><<<blocks, 128, 0, st>>>(a); break;
    default: return MS_ERR_ARG;
  }
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}
