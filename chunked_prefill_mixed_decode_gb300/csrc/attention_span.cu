// Mixed-batch attention over bf16 pools where a query does not see all keys up to
// its own: the last `window` of them, with an optional sink per head, or a fixed run of
// keys that no position bounds (the states of an encoder, of a length of their own).
//
//     out[t, h] = sum_j e^(s_j) V[j] / (e^(sink_h) + sum_j e^(s_j)),   j in the token's span
//
// The structure is the causal kernel's (attention.cu): a prologue, then one persistent CTA
// per SM over the decode and the chunk queue.  A decode row's items start at the page of its
// first key; an item of a chunk row walks the 64-key tiles from the page of its first
// query's first key to its last query's last key, and each of its two Q tiles only those
// that it sees.  Nothing of a row in front of that page is read, its table entries included.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attention_bf16.cuh"

namespace {

// Tensor maps of the chunk rows: K, V and both by groups of 8 keys, and the output.
struct SpanMaps {
  CUtensorMap k, v, kv, out;
};

// The cost model's SM time of a 128x128 chunk tile beside decode rows (attention_step.cuh): from sweeps of the split
// over eleven mixed steps, in a build that forced it for the purpose (256 decodes and two chunks of 3968 tokens over
// 1024 keys: 263 us at the causal kernel's 5820, 235 here; 100 decodes and 2000 tokens, D = 64, over 1500 keys 113
// and 103).
constexpr float kSpanTileCycles = 4000.f;

template <int D, int G>
__global__ void __launch_bounds__(kChunkThreads, 1)
    attention_span_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_vp,
                          const __grid_constant__ CUtensorMap tm_kp, const __grid_constant__ SpanMaps m, AttnParams p) {
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
  griddep_wait();  // the prologue's item tables (and, through it, what ran before it)
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
      chunk_phase<D, G, kSpan>(&tm_q, &m.k, &m.v, &m.kv, p, smem, tmem, &m.out);
      tc_fence_before();
      __syncthreads();
      ChBars* bars = reinterpret_cast<ChBars*>(smem + ChCfg<D>::BAR_OFF);
      const bool aborted = bars->abort != 0;
      if (threadIdx.x == 0) close_span_barriers(bars);
      __syncthreads();
      if (aborted) break;
    } else if (!chunk && n_dec_items > 0) {
      decode_phase<D, G, true>(p, smem, &tm_k, &tm_v, &tm_kp, &tm_vp);
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

template <int D, int G>
int launch_span(const AttnPlan& L, const SpanMaps& m, cudaStream_t st) {
  constexpr int chunk = ChCfg<D>::SMEM + kSoftmaxWarps * 4096;  // and the stages of store_rows
  constexpr int smem = chunk > DecCfg<D, G>::SMEM ? chunk : DecCfg<D, G>::SMEM;
  static_assert(smem <= 232448, "attention kernel exceeds the per-CTA shared-memory limit");
  const int slot = (D == 128 ? 4 : 0) + (G == 1 ? 0 : G == 2 ? 1 : G == 4 ? 2 : 3);  // one bit per instance
  if (ensure_smem_limit(attention_span_kernel<D, G>, slot, smem) != MS_OK) return MS_ERR_CUDA;
  if (launch_dependent(attention_span_kernel<D, G>, dim3(L.p.num_sms), dim3(kChunkThreads), smem, st, L.tq, L.tk, L.tv,
                       L.tvp, L.tkp, m, L.p) != cudaSuccess)
    return MS_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}

// Both calls: every argument check comes before the first enqueue.  window == 0: a fixed run of keys.
int span_call(const void* q, const void* k_cache, const void* v_cache, int32_t num_pages, const int32_t* cu_seqlens_q,
              const int32_t* q_start_pos, const int32_t* lens, const int32_t* block_tables, const int32_t* bt_offsets,
              int64_t bt_len, int32_t bt_stride, int32_t num_rows, int32_t num_tokens, int64_t key_total, int32_t H_q,
              int32_t H_kv, int32_t D, int32_t page_size, float scale, int32_t window, const float* sinks, void* out,
              void* workspace, size_t ws_bytes, int64_t stall_limit_ns, ms_stream_t stream) {
  if ((reinterpret_cast<uintptr_t>(sinks) & 3u) != 0) return MS_ERR_ARG;
  AttnPlan L;
  bool empty = true;
  int rc = attention_setup(q, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, lens, block_tables, bt_offsets,
                           bt_offsets != nullptr ? bt_len : 0, bt_offsets != nullptr ? 0 : bt_stride, num_rows, num_tokens,
                           key_total, H_q, H_kv, D, page_size, scale, out, workspace, ws_bytes, false, stall_limit_ns, &L,
                           &empty);
  if (rc != MS_OK || empty) return rc;
  L.p.tile_cycles = kSpanTileCycles;
  L.p.sinks = sinks;
  L.p.fixed_span = window == 0 ? 1 : 0;
  L.p.window = window == 0 ? INT32_MAX : window;
  set_parts_room(&L.p, workspace, ws_bytes, key_total);
  // K and V of the chunk tiles, by groups of 8 keys and 64-column slabs (SpanTile): maps of one pool, and of both
  // where the pools' distance is a stride that a map can have
  SpanMaps m;
  const EncodeTiledFn enc = get_encode_fn();
  const cuuint64_t slabs = static_cast<cuuint64_t>(D) / 64, groups = 2 * static_cast<cuuint64_t>(num_pages) * H_kv;
  const cuuint64_t row = static_cast<cuuint64_t>(D) * 2;
  {
    const cuuint64_t dims[4] = {64, 8, D == 128 ? slabs : groups, groups}, strides[3] = {row, D == 128 ? 128 : 8 * row, 8 * row};
    const cuuint32_t box[4] = {64, 8, 2, 2};
    const int rank = D == 128 ? 4 : 3;
    if (!encode_bf16(enc, &m.k, k_cache, rank, dims, strides, box) || !encode_bf16(enc, &m.v, v_cache, rank, dims, strides, box))
      return MS_ERR_ARG;
  }
  const uintptr_t ka = reinterpret_cast<uintptr_t>(k_cache), va = reinterpret_cast<uintptr_t>(v_cache);
  const uintptr_t apart = ka < va ? va - ka : ka - va;  // both 16-byte aligned
  m.kv = m.k;
  if (apart != 0 && apart < (uintptr_t{1} << 40)) {
    const void* low = ka < va ? k_cache : v_cache;
    const cuuint64_t dims5[5] = {64, 8, slabs, 2, groups}, strides5[4] = {row, 128, apart, 8 * row};
    const cuuint64_t dims4[4] = {64, 8, 2, groups}, strides4[3] = {row, apart, 8 * row};
    const cuuint32_t box[5] = {64, 8, 2, 2, 2};
    if (D == 128 ? encode_bf16(enc, &m.kv, low, 5, dims5, strides5, box) : encode_bf16(enc, &m.kv, low, 4, dims4, strides4, box))
      L.p.kv_form = ka < va ? kKvKFirst : kKvVFirst;
  }
  // 32 rows (32 / G tokens of G heads) of 64 columns of the output
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H_q), static_cast<cuuint64_t>(num_tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H_q) * D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(L.p.G), static_cast<cuuint32_t>(32 / L.p.G)};
  if (!encode_bf16(enc, &m.out, out, 3, dims, strides, box)) return MS_ERR_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  rc = launch_prologue<false, true>(L.p, st);
  if (rc != MS_OK) return rc;
  switch (D * 100 + L.p.G) {
    case 6401: return launch_span<64, 1>(L, m, st);
    case 6402: return launch_span<64, 2>(L, m, st);
    case 6404: return launch_span<64, 4>(L, m, st);
    case 6408: return launch_span<64, 8>(L, m, st);
    case 12801: return launch_span<128, 1>(L, m, st);
    case 12802: return launch_span<128, 2>(L, m, st);
    case 12804: return launch_span<128, 4>(L, m, st);
    default: return launch_span<128, 8>(L, m, st);
  }
}

}  // namespace

extern "C" MS_API int ms_mixed_step_attention_window(
    const void* q_rot, const void* k_cache, const void* v_cache, int32_t num_pages, const int32_t* cu_seqlens_q,
    const int32_t* q_start_pos, const int32_t* context_lens, const int32_t* block_tables, const int32_t* bt_offsets,
    int64_t bt_len, int32_t bt_stride, int32_t num_rows, int32_t num_tokens, int64_t context_total, int32_t H_q,
    int32_t H_kv, int32_t D, int32_t page_size, float scale, int32_t window, const float* sinks, void* out,
    void* workspace, size_t ws_bytes, ms_stream_t stream) {
  if (window < 1) return MS_ERR_ARG;
  return span_call(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables, bt_offsets,
                   bt_len, bt_stride, num_rows, num_tokens, context_total, H_q, H_kv, D, page_size, scale, window, sinks,
                   out, workspace, ws_bytes, 0, stream);
}

extern "C" MS_API int ms_mixed_step_cross_attention(
    const void* q, const void* k_cache, const void* v_cache, int32_t num_pages, const int32_t* cu_seqlens_q,
    const int32_t* key_lens, const int32_t* block_tables, const int32_t* bt_offsets, int64_t bt_len, int32_t bt_stride,
    int32_t num_rows, int32_t num_tokens, int64_t key_total, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
    float scale, void* out, void* workspace, size_t ws_bytes, ms_stream_t stream) {
  return span_call(q, k_cache, v_cache, num_pages, cu_seqlens_q, key_lens, key_lens, block_tables, bt_offsets, bt_len,
                   bt_stride, num_rows, num_tokens, key_total, H_q, H_kv, D, page_size, scale, 0, nullptr, out, workspace,
                   ws_bytes, 0, stream);
}

extern "C" MS_API int ms_test_attention_stall_window(
    const void* q_rot, const void* k_cache, const void* v_cache, int32_t num_pages, const int32_t* cu_seqlens_q,
    const int32_t* q_start_pos, const int32_t* context_lens, const int32_t* block_tables, int32_t bt_stride,
    int32_t num_rows, int32_t num_tokens, int64_t context_total, int32_t H_q, int32_t H_kv, int32_t D, int32_t page_size,
    float scale, int32_t window, void* out, void* workspace, size_t ws_bytes, int64_t wait_limit_ns, ms_stream_t stream) {
  if (window < 1 || wait_limit_ns < 100000 || wait_limit_ns > 2000000000ll) return MS_ERR_ARG;  // 0.1 ms .. 2 s
  return span_call(q_rot, k_cache, v_cache, num_pages, cu_seqlens_q, q_start_pos, context_lens, block_tables, nullptr, 0,
                   bt_stride, num_rows, num_tokens, context_total, H_q, H_kv, D, page_size, scale, window, nullptr, out,
                   workspace, ws_bytes, wait_limit_ns, stream);
}
