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
#include "attention_bf16.cuh"
#include "mixed_step.h"
#include "ptx.cuh"

namespace {

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
