// The step's metadata built on the GPU from the requests' lengths, so that a
// step (or a captured run of steps) needs no data from the host.
//
// Row s is request s, with c cached tokens and d new ones.  Three prefix sums
// over the rows carry everything: tokens (d), pages in use (ceil((c + d) / 16))
// and new pages (those minus ceil(c / 16)).  Every other output element then
// follows from its row and its offset within it, and the row from a binary
// search of a prefix; page j of a row is an entry of its page table while
// j < ceil(c / 16), and else the next one from the end of the free list.
//
// Every CTA scans all rows by itself (at most 8192, read from L2) and expands
// its share of the outputs, so nothing waits on another CTA and one launch is
// enough.  Only the free count may be read and written in place: the last CTA
// to finish, told by a counter, writes it.
//
// Bound by latency: the lengths' loads, the scan, a search of the prefix, a page's
// load, one after the other.  In a replayed graph 64 rows take 5.4 us; 513 rows of a
// long mixed step into a padded table of 16.8 MB 16.2 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "device_state.cuh"
#include "mixed_step.h"

namespace {

constexpr int kPage = 16;
constexpr int kMetaThreads = 512;
constexpr int kMetaMaxRows = 8192;
constexpr int kMetaMaxTokens = 1 << 21;

// 32-bit words of dynamic shared memory for R rows
constexpr int metadata_words(int R) { return 4 * (R + 1); }

struct MetaArgs {
  const int32_t* cached;
  const int32_t* fresh;
  int32_t* tables;
  const int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_state;
  int32_t* cu;
  int32_t* q_start;
  int32_t* ctx;
  int32_t* positions;
  int32_t* slots;
  int32_t* block_tables;
  int32_t* bt_offsets;
  int32_t* bt_pages;
  int32_t* info;
  int32_t* status;
  int64_t cap_pages;
  int32_t num_rows, table_stride, free_cap, num_pages, cap_tokens, bt_stride;
};

// pages of n >= 0 tokens
__device__ __forceinline__ int pages_of(int32_t n) {
  return static_cast<int>((static_cast<uint32_t>(n) + kPage - 1) / kPage);
}

// Rows whose spans of the prefix `p` (n + 1 entries) hold i[0..U): the last row
// with p[row] <= i, which skips empty rows.  U searches side by side, every one
// of the same number of steps, so that their shared-memory loads overlap.
template <int U>
__device__ __forceinline__ void rows_of(const int32_t* p, int n, const int (&i)[U], int (&row)[U]) {
#pragma unroll
  for (int j = 0; j < U; ++j) row[j] = 0;
  for (int step = 1 << (31 - __clz(n)); step > 0; step >>= 1) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int r = row[j] + step;
      if (r < n && p[r] <= i[j]) row[j] = r;
    }
  }
}

__device__ __forceinline__ int64_t warp_inclusive(int64_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

__global__ void __launch_bounds__(kMetaThreads) metadata_kernel(MetaArgs a) {
  extern __shared__ int32_t sm[];
  __shared__ int64_t s_warp[3][kMetaThreads / 32];
  __shared__ int s_dec;
  const int R = a.num_rows, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int32_t* s_tok = sm;             // prefix of tokens, R + 1 entries
  int32_t* s_pg = s_tok + R + 1;   // prefix of pages in use
  int32_t* s_new = s_pg + R + 1;   // prefix of new pages
  int32_t* s_c = s_new + R + 1;    // cached tokens
  if (tid == 0) s_dec = 0;
  const int fc = a.free_count != nullptr ? *a.free_count : 0;

  // 1. each thread's run of rows: sums and checks
  const int per = (R + kMetaThreads - 1) / kMetaThreads;
  const int r0 = min(R, tid * per), r1 = min(R, r0 + per);
  int64_t tok = 0, pg = 0, nw = 0;
  int decodes = 0, bad = 0;
  for (int r = r0; r < r1; ++r) {
    const int32_t c = a.cached[r], d = a.fresh[r];
    if (c < 0 || d < 0 || static_cast<int64_t>(c) + d > INT32_MAX) {
      bad |= MS_STATUS_BAD_META;
      continue;
    }
    if (d == 0) continue;  // a pad row: no tokens, no context, no pages
    const int held = pages_of(c);
    const int need = pages_of(c + d);
    if (need > a.table_stride) bad |= MS_STATUS_NO_PAGES;
    if (a.block_tables != nullptr && need > a.bt_stride) bad |= MS_STATUS_BAD_META;
    tok += d;
    pg += need;
    if (a.free_pages != nullptr) nw += need - held;
    decodes += d == 1;
  }
  const int64_t my_tok = tok, my_pg = pg, my_nw = nw;
  tok = warp_inclusive(tok);
  pg = warp_inclusive(pg);
  nw = warp_inclusive(nw);
  if (lane == 31) {
    s_warp[0][warp] = tok;
    s_warp[1][warp] = pg;
    s_warp[2][warp] = nw;
  }
  decodes = __reduce_add_sync(0xffffffffu, decodes);
  bad = __reduce_or_sync(0xffffffffu, bad);
  __syncthreads();
  if (lane == 0 && decodes > 0) atomicAdd(&s_dec, decodes);
  int64_t tot_tok = 0, tot_pg = 0, tot_new = 0, b_tok = 0, b_pg = 0, b_new = 0;
  for (int w = 0; w < kMetaThreads / 32; ++w) {
    if (w == warp) {
      b_tok = tot_tok;
      b_pg = tot_pg;
      b_new = tot_new;
    }
    tot_tok += s_warp[0][w];
    tot_pg += s_warp[1][w];
    tot_new += s_warp[2][w];
  }
  // checks of the totals: the same in every thread
  if (tot_tok > a.cap_tokens) bad |= MS_STATUS_BAD_META;
  if (tot_pg > INT32_MAX || (a.bt_pages != nullptr && tot_pg > a.cap_pages)) bad |= MS_STATUS_BAD_META;
  if (a.free_pages != nullptr) {
    if (fc < 0 || fc > a.free_cap) bad |= MS_STATUS_BAD_META;
    if (tot_new > fc) bad |= MS_STATUS_NO_PAGES;
  }
  // a step that fails a check becomes one of pad rows only
  const int bad_meta = __syncthreads_or(bad & MS_STATUS_BAD_META);
  const int no_pages = __syncthreads_or(bad & MS_STATUS_NO_PAGES);
  bad = (bad_meta ? MS_STATUS_BAD_META : 0) | (no_pages ? MS_STATUS_NO_PAGES : 0);
  if (bad) tot_tok = tot_pg = tot_new = 0;
  // 2. prefixes in shared memory; CTA 0 writes the rows
  int64_t o_tok = b_tok + tok - my_tok, o_pg = b_pg + pg - my_pg, o_new = b_new + nw - my_nw;
  for (int r = r0; r < r1; ++r) {
    const int32_t c = a.cached[r], d = bad ? 0 : a.fresh[r];
    s_c[r] = c;
    s_tok[r] = bad ? 0 : static_cast<int32_t>(o_tok);
    s_pg[r] = bad ? 0 : static_cast<int32_t>(o_pg);
    s_new[r] = bad ? 0 : static_cast<int32_t>(o_new);
    if (blockIdx.x == 0) {
      a.cu[r] = s_tok[r];
      a.q_start[r] = d > 0 ? c : 0;
      a.ctx[r] = d > 0 ? c + d : 0;
      if (a.bt_offsets != nullptr) a.bt_offsets[r] = s_pg[r];
    }
    if (d > 0) {
      const int held = pages_of(c);
      const int need = pages_of(c + d);
      o_tok += d;
      o_pg += need;
      if (a.free_pages != nullptr) o_new += need - held;
    }
  }
  if (tid == 0) {
    s_tok[R] = static_cast<int32_t>(tot_tok);
    s_pg[R] = static_cast<int32_t>(tot_pg);
    s_new[R] = static_cast<int32_t>(tot_new);
    if (blockIdx.x == 0) {
      a.cu[R] = static_cast<int32_t>(tot_tok);
      if (a.bt_offsets != nullptr) a.bt_offsets[R] = static_cast<int32_t>(tot_pg);
      if (a.info != nullptr) {
        a.info[0] = static_cast<int32_t>(tot_tok);
        a.info[1] = static_cast<int32_t>(tot_pg);
        a.info[2] = bad ? 0 : s_dec;
        a.info[3] = static_cast<int32_t>(tot_new);
      }
      if (bad && a.status != nullptr) atomicOr(a.status, bad);
    }
  }
  __syncthreads();

  // page j of row r, of its `held` old pages or of the new ones after them
  auto page_at = [&](int r, int j) -> int32_t {
    const int fresh = s_new[r + 1] - s_new[r], held = s_pg[r + 1] - s_pg[r] - fresh;
    const int32_t* src = j < held || fresh == 0 ? a.tables + static_cast<int64_t>(r) * a.table_stride + j
                                                : a.free_pages + (fc - 1 - (s_new[r] + j - held));
    return *src;
  };
  // the CTA's elements of an output, U to a thread at a time
  constexpr int U = 4;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kMetaThreads * U + tid;
  const int64_t first_tok = static_cast<int64_t>(gridDim.x - 1 - blockIdx.x) * kMetaThreads * U + tid;  // from the other end
  const int64_t gstride = static_cast<int64_t>(gridDim.x) * kMetaThreads * U;
  // 3. tokens; those past the total are pad tokens (position 0, no slot)
  for (int64_t t0 = first_tok; t0 < a.cap_tokens; t0 += gstride) {
    int t[U], r[U], pos[U], page[U];
#pragma unroll
    for (int j = 0; j < U; ++j) t[j] = static_cast<int>(min(t0 + j * kMetaThreads, static_cast<int64_t>(kMetaMaxTokens)));
    rows_of<U>(s_tok, R, t, r);
#pragma unroll
    for (int j = 0; j < U; ++j) {
      pos[j] = 0;
      page[j] = -1;
      if (t[j] < tot_tok) {
        pos[j] = s_c[r[j]] + t[j] - s_tok[r[j]];
        page[j] = page_at(r[j], pos[j] / kPage);
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (t[j] >= a.cap_tokens) continue;
      const bool ok = page[j] >= 0 && page[j] < a.num_pages;
      if (!ok && t[j] < tot_tok && a.status != nullptr) atomicOr(a.status, MS_STATUS_BAD_PAGE);
      a.positions[t[j]] = pos[j];
      a.slots[t[j]] = ok ? page[j] * kPage + pos[j] % kPage : -1;
    }
  }
  // 4. the block table
  if (a.bt_pages != nullptr) {
    for (int64_t i0 = first; i0 < tot_pg; i0 += gstride) {
      int i[U], r[U], page[U];
#pragma unroll
      for (int j = 0; j < U; ++j) i[j] = static_cast<int>(min(i0 + j * kMetaThreads, tot_pg - 1));
      rows_of<U>(s_pg, R, i, r);
#pragma unroll
      for (int j = 0; j < U; ++j) page[j] = page_at(r[j], i[j] - s_pg[r[j]]);
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i0 + j * kMetaThreads < tot_pg) a.bt_pages[i[j]] = page[j];
    }
  } else {
    const int64_t n = static_cast<int64_t>(R) * a.bt_stride;
    for (int64_t i0 = first; i0 < n; i0 += gstride) {
      int32_t page[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t i = min(i0 + j * kMetaThreads, n - 1);
        const int r = static_cast<int>(i / a.bt_stride), c = static_cast<int>(i - static_cast<int64_t>(r) * a.bt_stride);
        page[j] = c < s_pg[r + 1] - s_pg[r] ? page_at(r, c) : -1;
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (i0 + j * kMetaThreads < n) a.block_tables[i0 + j * kMetaThreads] = page[j];
    }
  }
  // An attention call directly after this one starts its prologue, which reads the rows, as soon as every
  // CTA here has ended: what the CTA wrote is performed by then.
  __threadfence();
  // 5. the new pages into the requests' tables, and the free count
  if (a.free_pages == nullptr) return;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kMetaThreads + tid; i0 < tot_new;
       i0 += static_cast<int64_t>(gridDim.x) * kMetaThreads) {
    const int i[1] = {static_cast<int>(i0)};
    int r[1];
    rows_of<1>(s_new, R, i, r);
    a.tables[static_cast<int64_t>(r[0]) * a.table_stride + pages_of(s_c[r[0]]) + (i[0] - s_new[r[0]])] =
        a.free_pages[fc - 1 - i[0]];
  }
  __syncthreads();
  if (tid == 0) {
    // every thread of the CTA has used the count it read; the counter wraps to 0 by itself, ready for
    // the next call
    if (atomicInc(reinterpret_cast<unsigned*>(a.free_state + 1), gridDim.x - 1) == gridDim.x - 1)
      a.free_state[0] = fc - static_cast<int32_t>(tot_new);
  }
}

struct Span {
  const int32_t* p;
  int64_t n;
};

inline bool overlap(const Span& x, const Span& y) {
  return x.p != nullptr && y.p != nullptr && x.n > 0 && y.n > 0 && x.p < y.p + y.n && y.p < x.p + x.n;
}

}  // namespace

extern "C" MS_API int ms_build_batch_metadata_device(
    const int32_t* cached_lens, const int32_t* new_tokens, int32_t num_rows, int32_t* page_tables, int32_t table_stride,
    const int32_t* free_pages, int32_t free_cap, const int32_t* free_count, int32_t* free_state, int32_t num_pages,
    int32_t cap_tokens, int32_t* cu_seqlens_q, int32_t* q_start_pos, int32_t* context_lens, int32_t* positions,
    int32_t* slot_mapping, int32_t* block_tables, int32_t bt_stride, int32_t* bt_offsets, int32_t* bt_pages,
    int64_t cap_pages, int32_t* info, int32_t* dev_status, ms_stream_t stream) {
  if (num_rows < 1 || num_rows > kMetaMaxRows || table_stride < 1 || cap_tokens < 0 || cap_tokens > kMetaMaxTokens ||
      num_pages < 0 || num_pages > INT32_MAX / kPage || free_cap < 0)
    return MS_ERR_ARG;
  if (!cached_lens || !new_tokens || !page_tables || !cu_seqlens_q || !q_start_pos || !context_lens) return MS_ERR_ARG;
  if (cap_tokens > 0 && (!positions || !slot_mapping)) return MS_ERR_ARG;
  const bool ragged = bt_offsets != nullptr;
  if (ragged ? (block_tables != nullptr || !bt_pages || cap_pages < 0) : (!block_tables || bt_pages || bt_stride < 1))
    return MS_ERR_ARG;
  const bool alloc = free_pages != nullptr;
  if (alloc != (free_count != nullptr) || alloc != (free_state != nullptr)) return MS_ERR_ARG;
  // the kernel's CTAs read the inputs while others write the outputs
  const int64_t R = num_rows, table_n = ragged ? cap_pages : R * bt_stride;
  const Span in[] = {{cached_lens, R}, {new_tokens, R}, {page_tables, R * table_stride}, {free_pages, free_cap}};
  const Span out[] = {{cu_seqlens_q, R + 1}, {q_start_pos, R}, {context_lens, R}, {positions, cap_tokens},
                      {slot_mapping, cap_tokens}, {ragged ? bt_pages : block_tables, table_n}, {bt_offsets, R + 1},
                      {info, 4}};
  const Span status{dev_status, 1}, state{free_state, 2}, count{free_count, 1};
  for (const Span& x : in) {
    if (overlap(x, status) || overlap(x, state)) return MS_ERR_ARG;
    for (const Span& y : out)
      if (overlap(x, y)) return MS_ERR_ARG;
  }
  // the free count is an input (written, with free_state's first word, only after every CTA has read it),
  // and the counter beside it lasts from call to call
  for (const Span& y : out)
    if (overlap(count, y) || overlap(state, y)) return MS_ERR_ARG;
  if (overlap(in[2], in[3]) || overlap(in[2], count) || overlap(status, count) || overlap(status, state) ||
      (alloc && free_count == free_state + 1))
    return MS_ERR_ARG;
  MetaArgs a{cached_lens, new_tokens, page_tables, free_pages, free_count, free_state, cu_seqlens_q, q_start_pos,
             context_lens, positions, slot_mapping, block_tables, bt_offsets, bt_pages, info, dev_status,
             cap_pages, num_rows, table_stride, free_cap, num_pages, cap_tokens, bt_stride};
  // 48 KB without a raised limit cover the kernel's static arrays too, so it is raised for every call
  if (ensure_smem_limit(metadata_kernel, 0, metadata_words(kMetaMaxRows) * 4) != MS_OK) return MS_ERR_CUDA;
  const int smem = metadata_words(num_rows) * 4;
  const int64_t most = table_n > cap_tokens ? table_n : cap_tokens;
  const int sms = ms_num_sms();
  if (sms <= 0) return MS_ERR_CUDA;
  int64_t blocks = (most + 4 * kMetaThreads - 1) / (4 * kMetaThreads);
  blocks = blocks < 1 ? 1 : blocks > 2 * sms ? 2 * sms : blocks;  // every CTA scans the rows: no more than run at once
  metadata_kernel<<<static_cast<unsigned>(blocks), kMetaThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? MS_OK : MS_ERR_CUDA;
}
